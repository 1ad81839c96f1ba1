"""Float64 CPU oracle for tree-verify MLA attention (test infrastructure).

TEST INFRASTRUCTURE ONLY: the tests, ``__graft_entry__.smoke()`` and the
benchmark's CPU-baseline leg are the only callers. The library's product path
never imports this package, and this package imports nothing from the library.

The arithmetic lives in ``mla_oracle.c`` (plain loops, float64, OpenMP over
rows); this module compiles it with gcc and marshals numpy arrays through
ctypes. See the C file's header for the definition it follows.
"""
from __future__ import annotations

import ctypes
import os
import subprocess
from typing import Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
_SRC = os.path.join(_HERE, "mla_oracle.c")
_LIB = os.path.join(_HERE, "libmla_oracle.so")
_lib = None

ERRORS = {0: "ok", -1: "invalid argument", -2: "tree parent out of order", -3: "slot out of range",
          -4: "out of memory"}


def build(force: bool = False) -> str:
    """Compile the oracle with gcc (portable flags: the same source builds on x86-64 and aarch64)."""
    if force or not os.path.exists(_LIB) or os.path.getmtime(_LIB) < os.path.getmtime(_SRC):
        tmp = _LIB + f".tmp{os.getpid()}"
        subprocess.run(["gcc", "-O2", "-std=c11", "-fopenmp", "-fPIC", "-shared", "-Wall", "-Wextra",
                        "-o", tmp, _SRC, "-lm"], check=True)
        os.replace(tmp, _LIB)
    return _LIB


def build_mutant(mutation: int, out_dir: str) -> str:
    """Compile a planted-mistake build (``-DORACLE_MUTATION=n``) into ``out_dir``; for the pin tests."""
    path = os.path.join(out_dir, f"libmla_oracle_mut{mutation}.so")
    subprocess.run(["gcc", "-O2", "-std=c11", "-fopenmp", "-fPIC", "-shared", f"-DORACLE_MUTATION={mutation}",
                    "-o", path, _SRC, "-lm"], check=True)
    return path


def _declare(lib):
    P = ctypes.c_void_p
    i32, i64, f64 = ctypes.c_int32, ctypes.c_int64, ctypes.c_double
    lib.oracle_verify.argtypes = [i32, i32, i32, i32, i32, P, P, i64, P, P, P, i64, f64, P, i64,
                                  i64, i64, P, P, i32]
    lib.oracle_verify.restype = ctypes.c_int
    lib.oracle_row_weights.argtypes = [i32, i32, i32, i32, i32, P, P, i64, P, P, P, i64, f64, i64, P]
    lib.oracle_row_weights.restype = ctypes.c_int
    lib.oracle_combine.argtypes = [i32, i64, i32, P, P, P, P]
    lib.oracle_combine.restype = ctypes.c_int
    lib.oracle_ancestor_masks.argtypes = [i32, P, P]
    lib.oracle_ancestor_masks.restype = ctypes.c_int
    lib.oracle_max_threads.restype = ctypes.c_int
    return lib


_active = None  # a planted-mistake library installed by the pin tests, else None


class use_library:
    """Context manager: route every oracle call through the library at ``path`` (pin tests only)."""

    def __init__(self, path: str):
        self.lib = _declare(ctypes.CDLL(path))

    def __enter__(self):
        global _active
        self.prev, _active = _active, self.lib
        return self

    def __exit__(self, *exc):
        global _active
        _active = self.prev


def _load():
    global _lib
    if _active is not None:
        return _active
    if _lib is None:
        build()
        lib = ctypes.CDLL(_LIB)
        _lib = _declare(lib)
    return _lib


def _ptr(a: np.ndarray):
    return a.ctypes.data_as(ctypes.c_void_p)


def _check(rc: int):
    if rc != 0:
        raise ValueError(f"oracle error {rc}: {ERRORS.get(rc, 'unknown')}")


def max_threads() -> int:
    return int(_load().oracle_max_threads())


def ancestor_masks(parent: np.ndarray) -> np.ndarray:
    parent = np.ascontiguousarray(parent, dtype=np.int32)
    out = np.zeros(len(parent), dtype=np.uint64)
    _check(_load().oracle_ancestor_masks(len(parent), _ptr(parent), _ptr(out)))
    return out


def verify(seq_lens, slot_table, tree_parent, q, kv, *, num_heads: int, scale: float,
           d_latent: int = 512, d_rope: int = 64, rows: Optional[Sequence[int]] = None,
           pos_begin: int = 0, pos_end: int = 2 ** 62, num_threads: int = 0):
    """Exact attention in float64. Returns (out [rows, d_latent], lse [rows]).

    ``q``: uint16 bf16 bits [B*T, H, d_latent + d_rope]; ``kv``: uint16 [num_slots, d_latent + d_rope];
    ``slot_table``: int32 [B, stride]; ``tree_parent``: int32 [B, T]; ``seq_lens``: int32 [B] prefix lengths.
    ``rows``: global row ids ``(b*T + i)*H + h`` (default all, in order).
    """
    seq_lens = np.ascontiguousarray(seq_lens, dtype=np.int32)
    slot_table = np.ascontiguousarray(slot_table, dtype=np.int32)
    tree_parent = np.ascontiguousarray(tree_parent, dtype=np.int32)
    q = np.ascontiguousarray(q, dtype=np.uint16)
    kv = np.ascontiguousarray(kv, dtype=np.uint16)
    B = len(seq_lens)
    T = tree_parent.shape[-1]
    H = num_heads
    dk = d_latent + d_rope
    assert q.size == B * T * H * dk and kv.shape[-1] == dk
    assert tree_parent.shape == (B, T) and slot_table.shape[0] == B
    if rows is None:
        rows_arr = None
        n = B * T * H
    else:
        rows_arr = np.ascontiguousarray(rows, dtype=np.int64)
        n = len(rows_arr)
    out = np.zeros((n, d_latent), dtype=np.float64)
    lse = np.zeros(n, dtype=np.float64)
    _check(_load().oracle_verify(B, T, H, d_latent, d_rope, _ptr(seq_lens), _ptr(slot_table),
                                 slot_table.shape[1], _ptr(tree_parent), _ptr(q), _ptr(kv),
                                 kv.shape[0], float(scale),
                                 _ptr(rows_arr) if rows_arr is not None else None, n,
                                 int(pos_begin), int(pos_end), _ptr(out), _ptr(lse), int(num_threads)))
    return out, lse


def row_weights(seq_lens, slot_table, tree_parent, q, kv, row: int, *, num_heads: int, scale: float,
                d_latent: int = 512, d_rope: int = 64) -> np.ndarray:
    """Softmax weights of one row over logical positions 0..N_b-1 (0 where not visible)."""
    seq_lens = np.ascontiguousarray(seq_lens, dtype=np.int32)
    slot_table = np.ascontiguousarray(slot_table, dtype=np.int32)
    tree_parent = np.ascontiguousarray(tree_parent, dtype=np.int32)
    q = np.ascontiguousarray(q, dtype=np.uint16)
    kv = np.ascontiguousarray(kv, dtype=np.uint16)
    B, T = tree_parent.shape
    b = row // num_heads // T
    w = np.zeros(int(seq_lens[b]) + T, dtype=np.float64)
    _check(_load().oracle_row_weights(B, T, num_heads, d_latent, d_rope, _ptr(seq_lens), _ptr(slot_table),
                                      slot_table.shape[1], _ptr(tree_parent), _ptr(q), _ptr(kv),
                                      kv.shape[0], float(scale), int(row), _ptr(w)))
    return w


def combine(part_o: np.ndarray, part_lse: np.ndarray):
    """Merge partials [S, rows, d_v] / [S, rows] into (out [rows, d_v], lse [rows]), float64."""
    part_o = np.ascontiguousarray(part_o, dtype=np.float64)
    part_lse = np.ascontiguousarray(part_lse, dtype=np.float64)
    S, rows, d_v = part_o.shape
    out = np.zeros((rows, d_v), dtype=np.float64)
    lse = np.zeros(rows, dtype=np.float64)
    _check(_load().oracle_combine(S, rows, d_v, _ptr(part_o), _ptr(part_lse), _ptr(out), _ptr(lse)))
    return out, lse


def verify_problem(p, scale: float, rows=None, **kw):
    """``verify`` on a seeded problem object (fields seq_lens, slot_table, tree_parent, q, kv, H)."""
    return verify(p.seq_lens, p.slot_table, p.tree_parent, p.q, p.kv, num_heads=p.H, scale=scale,
                  rows=rows, **kw)


# ---------------------------------------------------------------------------------------------
# KV-pool steps around verification (plain numpy, the definitions written out). They follow
# "The Moment of Certainty", The Final Piece (the tree nodes' rows live at their own slots,
# and accepted nodes are scattered, so accepting a path rewrites the slot table) and "The Moment
# of Reckoning (User Challenge...)", Output, item 4 (Tier-0 defragmentation keeps each request's
# KV contiguous in the pool).

def tree_kv_append(pool: np.ndarray, tree_kv: np.ndarray, slot_table: np.ndarray, seq_lens: np.ndarray,
                   num_nodes: int) -> np.ndarray:
    """pool[slot_table[b][L_b + j]] = tree_kv[b*T + j]; returns the new pool (the input is not modified)."""
    out = pool.copy()
    for b in range(len(seq_lens)):
        L = int(seq_lens[b])
        for j in range(num_nodes):
            out[int(slot_table[b, L + j])] = tree_kv[b * num_nodes + j]
    return out


def tree_accept_commit(slot_table: np.ndarray, seq_lens: np.ndarray, tree_parent: np.ndarray,
                       accepted: np.ndarray, num_accepted: np.ndarray, max_seq_len: int):
    """Accepted path first (in path order) behind the prefix, then the rejected nodes in node order;
    seq_lens += n. An invalid path (not root-first along parent links, n outside [0, T], or a prefix
    longer than max_seq_len) leaves the sequence unchanged. Returns (table, lens, valid per sequence)."""
    table = slot_table.copy()
    lens = seq_lens.copy()
    T = tree_parent.shape[1]
    valid = np.zeros(len(seq_lens), dtype=bool)
    for b in range(len(seq_lens)):
        L, n = int(seq_lens[b]), int(num_accepted[b])
        if not (0 <= L <= max_seq_len and 0 <= n <= T and L + n <= max_seq_len):
            continue
        path = [int(a) for a in accepted[b, :n]]
        ok = all(0 <= a < T for a in path) and len(set(path)) == n
        if ok:
            for k, a in enumerate(path):
                if int(tree_parent[b, a]) != (path[k - 1] if k else -1):
                    ok = False
        if not ok:
            continue
        old = [int(x) for x in slot_table[b, L:L + T]]
        order = path + [j for j in range(T) if j not in path]
        for pos, node in enumerate(order):
            table[b, L + pos] = old[node]
        lens[b] = L + n
        valid[b] = True
    return table, lens, valid


def kv_compact(src_pool: np.ndarray, slot_table: np.ndarray, seq_lens: np.ndarray, num_nodes: int,
               dst_base: np.ndarray, dst_slots: int):
    """dst[dst_base[b] + t] = src[slot_table[b][t]] and new_table[b][t] = dst_base[b] + t for
    t < L_b + T; rows of dst outside every range stay zero. Returns (dst, new_table)."""
    dst = np.zeros((dst_slots,) + src_pool.shape[1:], dtype=src_pool.dtype)
    table = slot_table.copy()
    for b in range(len(seq_lens)):
        for t in range(int(seq_lens[b]) + num_nodes):
            d = int(dst_base[b]) + t
            dst[d] = src_pool[int(slot_table[b, t])]
            table[b, t] = d
    return dst, table


# ---------------------------------------------------------------------------------------------
# The pool held in 4 bits and the slot maps (plain numpy, the definitions written out). A 416-byte row:
# 512 e2m1 codes (two to a byte, the even dim low), 32 e4m3 scales (one to 16 dims), 64 bf16 RoPE dims.

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127])


def _nearest_code(x: np.ndarray, grid: np.ndarray) -> np.ndarray:
    """Index of the value of an ascending grid nearest to each x >= 0; the even index at a tie."""
    i = np.clip(np.searchsorted(grid, x, side="right"), 1, len(grid) - 1)
    below, above = x - grid[i - 1], grid[i] - x
    return np.where((above < below) | ((above == below) & (i % 2 == 0)), i, i - 1)


def _bf16_values(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def kv4_quantise(bits: np.ndarray) -> np.ndarray:
    """bf16 rows (uint16 bits [n, 576]) as rows of the 4-bit pool (uint8 [n, 416])."""
    n = bits.shape[0]
    x = _bf16_values(np.ascontiguousarray(bits[:, :512])).reshape(n, 32, 16)
    out = np.zeros((n, 416), dtype=np.uint8)
    fine = np.isfinite(x).all(axis=2)
    top = np.where(fine, np.abs(np.where(np.isfinite(x), x, 0)).max(axis=2), 0)
    scale = _nearest_code(np.minimum(top / 6, 448), E4M3)
    s = E4M3[scale][:, :, None]
    y = np.where(fine[:, :, None] & (s > 0), np.where(np.isfinite(x), x, 0) / np.where(s > 0, s, 1), 0)
    code = _nearest_code(np.minimum(np.abs(y), 6), E2M1) + 8 * np.signbit(y)
    code = code.reshape(n, 256, 2).astype(np.uint8)
    out[:, :256] = code[:, :, 0] | (code[:, :, 1] << 4)
    out[:, 256:288] = np.where(fine, scale, 127)
    out[:, 288:] = np.ascontiguousarray(bits[:, 512:]).view(np.uint8).reshape(n, 128)
    return out


def kv4_values(rows: np.ndarray) -> np.ndarray:
    """Rows of the 4-bit pool (uint8 [n, 416]) as the values they stand for (float64 [n, 576])."""
    n = rows.shape[0]
    out = np.empty((n, 576))
    for k in (0, 1):
        c = (rows[:, :256] >> (4 * k)) & 15
        out[:, k:512:2] = np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7]
    s = rows[:, 256:288]
    s = np.where((s & 127) == 127, np.nan, np.where(s >= 128, -1.0, 1.0) * E4M3[np.minimum(s & 127, 126)])
    out[:, :512] *= np.repeat(s, 16, axis=1)
    out[:, 512:] = _bf16_values(np.ascontiguousarray(rows[:, 288:]).view(np.uint16))
    return out


def kv4_bf16(rows: np.ndarray) -> np.ndarray:
    """The same values as bf16 bits (uint16 [n, 576]): every one of them is a bf16 number."""
    v = kv4_values(rows).astype(np.float32)
    bits = v.view(np.uint32)
    assert ((bits & 0xFFFF) == 0)[np.isfinite(v)].all()
    return (bits >> 16).astype(np.uint16)


def slot_map_build(seq_lens, new_lens, held_lens, page_size: int, num_pages: int, free_pages, free_count: int,
                   block_table, slot_table, map_capacity: int):
    """The definition of mla_slot_map_build, sequence by sequence. Returns (block_table, slot_table, slot_map,
    cu_new, held_out, free_left, bits) with bits a set of "length", "pages" and "slot" findings; inputs are not modified."""
    B, p = len(seq_lens), page_size
    held_lens = seq_lens if held_lens is None else held_lens
    block, table = None if block_table is None else block_table.copy(), slot_table.copy()
    slot_map = np.full(map_capacity, -1, dtype=np.int32)
    found, wish = set(), []
    for b in range(B):
        L, n, h = int(seq_lens[b]), int(new_lens[b]), int(held_lens[b])
        end = max(h, L + n)
        if L < 0 or n < 0 or h < L or end > table.shape[1] or (block is not None and -(-end // p) > block.shape[1]):
            found.add("length")
            n, end = 0, h
            wish.append((L, n, h, end, 0))
        else:
            wish.append((L, n, h, end, -(-end // p) - -(-h // p)))
    tokens, take = sum(w[1] for w in wish), sum(w[4] for w in wish)
    if tokens > map_capacity or not 0 <= free_count <= len(free_pages) or take > free_count:
        found.add("pages")
        return (block, table, slot_map, np.zeros(B + 1, np.int32), np.array([w[2] for w in wish], np.int32), free_count, found)
    cu, left = [0], free_count
    for b, (L, n, h, end, take) in enumerate(wish):
        have = -(-h // p)
        pages = [int(free_pages[left - 1 - k]) for k in range(take)]
        left -= take
        if block is not None:
            block[b, have:have + take] = pages
        for t in range(L, L + n):
            if t < h:
                slot = int(table[b, t])
                bad = not 0 <= slot < num_pages * p
            else:
                page = pages[t // p - have] if t // p >= have else int(block[b, t // p])
                slot, bad = page * p + t % p, not 0 <= page < num_pages
            if bad:
                found.add("slot")
                slot = -1
            if t >= h:
                table[b, t] = slot
            slot_map[cu[-1] + t - L] = slot
        cu.append(cu[-1] + n)
    return (block, table, slot_map, np.array(cu, np.int32), np.array([w[3] for w in wish], np.int32), left, found)


# ---- a layer's norms and rotations, and prompt attention, as include/mla_prompt.h defines them ----
def turn(x: np.ndarray, cos_sin: np.ndarray, halves: bool) -> np.ndarray:
    """Vectors [n, ..., 64] (float64), token i turned by cos_sin[i] = 32 cosines, 32 sines."""
    c = cos_sin[:, :32].astype(np.float64).reshape((-1,) + (1,) * (x.ndim - 2) + (32,))
    s = cos_sin[:, 32:].astype(np.float64).reshape(c.shape)
    a = np.arange(32) if halves else 2 * np.arange(32)
    b = a + (32 if halves else 1)
    y = np.empty_like(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def norm(x: np.ndarray, weight: Optional[np.ndarray], eps: float) -> np.ndarray:
    """weight * x / sqrt(mean(x^2) + eps) over the last axis (x itself without a weight)."""
    return x if weight is None else weight * x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def rope_rows(rows: np.ndarray, cos_sin: np.ndarray, weight: Optional[np.ndarray], eps: float, halves: bool) -> np.ndarray:
    """rows [n, 576] in float64: the latent dims normalised, the RoPE dims turned."""
    return np.concatenate([norm(rows[:, :512], weight, eps), turn(rows[:, 512:], cos_sin, halves)], 1)


def rope_heads(q: np.ndarray, cos_sin: np.ndarray, weight: Optional[np.ndarray], eps: float, halves: bool) -> np.ndarray:
    """Query heads [n, heads, d] in float64: normalised, their last 64 dims turned."""
    z = norm(q, weight, eps)
    return np.concatenate([z[..., :-64], turn(z[..., -64:], cos_sin, halves)], -1)


def prompt_attn(q, k, k_rope, v, cu_q, cu_k, *, causal: bool, scale: float):
    """(out, lse, spread, size) in float64: spread = sum of weights times |values|, size = the largest sum of |q||k| among
    the keys that a row sees, times scale (what a rounding error of the scores is relative to). Rows outside the
    sequences stay NaN; a row without keys has out 0, lse -inf."""
    heads, group = q.shape[1], q.shape[1] // k.shape[1]
    out = np.full((q.shape[0], heads, v.shape[2]), np.nan)
    spread, lse, size = out.copy(), np.full((q.shape[0], heads), np.nan), np.full((q.shape[0], heads), np.nan)
    for b in range(len(cu_q) - 1):
        m, n = int(cu_q[b + 1] - cu_q[b]), int(cu_k[b + 1] - cu_k[b])
        if m == 0:
            continue
        at = slice(int(cu_k[b]), int(cu_k[b]) + n)
        for h in range(heads):
            key = np.concatenate([k[at, h // group], k_rope[at]], 1)
            val = v[at, h // group]
            rows = q[int(cu_q[b]):int(cu_q[b]) + m, h]
            with np.errstate(invalid="ignore", over="ignore"):
                s, mag = rows @ key.T * scale, np.abs(rows) @ np.abs(key).T * scale
                for i in range(m):
                    r, vis = int(cu_q[b]) + i, max(0, min(n, i + n - m + 1)) if causal else n
                    if vis == 0:
                        out[r, h], spread[r, h], lse[r, h], size[r, h] = 0.0, 0.0, -np.inf, 0.0
                        continue
                    top = s[i, :vis].max()
                    w = np.exp(s[i, :vis] - top)
                    z = w.sum()
                    out[r, h], spread[r, h] = w / z @ val[:vis], w / z @ np.abs(val[:vis])
                    lse[r, h], size[r, h] = top + np.log(z), mag[i, :vis].max()
    return out, lse, spread, size
