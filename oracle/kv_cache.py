"""Plain NumPy implementation of the quantized KV cache (test infrastructure):
page tables from lengths, quantized appending, causal attention.

["Infra Quant II", QuaRot Method: per-head Hadamard of queries and keys, cache
quantization, attention over dequantized blocks.] Written from the definitions
in include/rotw4a4.h, request by request; shares no code with the GPU path.
"""
from __future__ import annotations

import numpy as np

F32_MAX = np.finfo(np.float32).max


def _pages(n: int, page: int) -> int:
    return -(-n // page)


def kv_plan(ctx, new, table, free, n_free, T, page, capacity=None):
    """Returns a dict of every output; the inputs are not changed."""
    B, width = table.shape
    table, free = table.copy(), free.copy()
    cap = len(free)
    stack = list(free[:min(max(int(n_free), 0), cap)])
    low = len(stack)
    cu, status, first = [0], [], []
    for b in range(B):
        c, n = int(ctx[b]), int(new[b])
        end = cu[-1] + max(n, 0)
        bad = c < 0 or c > width * page or n < -1 or c + max(n, 0) > width * page or end > T
        status.append(2 if bad else 0)
        cu.append(end)
    for b in range(B):                                  # pages of ended requests
        if status[b] == 0 and new[b] == -1:
            stack += list(table[b, :_pages(int(ctx[b]), page)])
    stack = stack[:cap]
    free[low:len(stack)] = stack[low:]
    refused = False
    kv = np.zeros(B, np.int32)
    slot, pos = np.full(T, -1, np.int64), np.full(T, -1, np.int32)
    for b in range(B):
        c, n = int(ctx[b]), int(new[b])
        if status[b] == 2 or n == -1:
            continue
        had = _pages(c, page)
        need = _pages(c + n, page) - had
        if need > 0 and (refused or need > len(stack)):
            status[b], refused = 1, True
            continue
        for i in range(need):
            table[b, had + i] = stack.pop()
        kv[b] = c + n
        for i in range(n):
            p = c + i
            pos[cu[b] + i] = p
            slot[cu[b] + i] = int(table[b, p // page]) * page + p % page
    return {"cu_new": np.minimum(np.array(cu), T).astype(np.int32), "kv_len": kv, "slot": slot,
            "pos": pos, "status": np.array(status, np.int32),
            "n_free": np.array([len(stack)], np.int32), "page_table": table, "free_pages": free}


def kv_ctx_next(ctx, plan):
    """The next step's lengths: those of the plan, but what it does not serve stays."""
    return np.where(plan["status"] == 0, plan["kv_len"], ctx).astype(np.int32)


def hadamard_rows(x):
    """Normalized Hadamard transform of the last axis in x's own type, strides
    1, 2, 4, ... and one multiply at the end."""
    n, h = x.shape[-1], 1
    while h < n:
        y = x.reshape(x.shape[:-1] + (n // (2 * h), 2, h))
        a, b = y[..., 0, :], y[..., 1, :]
        x = np.stack([a + b, a - b], -2).reshape(x.shape)
        h *= 2
    return x * x.dtype.type(1.0 / np.sqrt(n))


def _append_one(x, codes, scale, cu, slot, rotate):
    H, page, dh = codes.shape[1:]
    x = x.astype(np.float32).reshape(len(x), H, dh)
    with np.errstate(all="ignore"):
        x = hadamard_rows(x) if rotate else x
    x = np.clip(np.where(np.isnan(x), np.float32(0), x), -F32_MAX, F32_MAX)
    for b in range(len(cu) - 1):
        t = int(cu[b])
        while t < cu[b + 1]:
            if slot[t] < 0:
                t += 1
                continue
            p, off = divmod(int(slot[t]), page)
            n = min(page - off, int(cu[b + 1]) - t)
            rows = x[t:t + n]
            t += n
            if p >= len(codes):
                continue
            old = scale[p] if off else np.zeros(H, np.float32)
            s = np.maximum(old, np.abs(rows).max((0, 2)) / np.float32(127))
            d = np.where(s > 0, s, np.float32(1))
            r = (old / d).astype(np.float32)
            again = np.rint(codes[p, :, :off].astype(np.float32) * r[:, None, None])
            codes[p, :, :off] = again.astype(np.int8)
            with np.errstate(over="ignore"):
                q = np.clip(np.rint(rows / d[None, :, None]), -127, 127)
            codes[p, :, off:off + n] = q.transpose(1, 0, 2).astype(np.int8)
            scale[p] = s


def kv_append(k, v, cache, cu, slot, rotate=False):
    """k, v float32 [T][H * dh]; cache a tuple of arrays, changed in place."""
    _append_one(k, cache[0], cache[1], cu, slot, rotate)
    _append_one(v, cache[2], cache[3], cu, slot, False)


def kv_attention(q, cache, table, cu, kv_len, scale, rotate=False, q_rounded=False):
    """(out float64 [T][Hq * dh], tolerance of the same shape).

    The tolerance follows from the roundings the kernel is allowed, for a row
    with n keys, weights p_j (sum 1) and A = sum_j p_j |v_j| per column:
      * bf16 output: 2^-8 |o|;
      * fp16 weights: 2^-11 A, and below fp16's normal range half a step, 2^-25
        in fp16. A weight carries its page's value scale relative to the largest
        scale S_v among the pages of the row's own keys, and stands for at least
        2^7 where it is the largest: n 2^-32 127 S_v, as codes are within 127;
      * scores in fp32: dh + 8 roundings of 2^-24 of S = max_j scale sum_d
        |q_d k_jd|; with queries rounded to fp16 (q_rounded: fp32 or transformed
        ones) 2^-11 S more. With errors of the scores of at most e, p_j =
        exp(s_j) / sum_i exp(s_i) changes by a factor within exp(-2 e) and
        exp(2 e), so o by (exp(2 e) - 1) A;
      * the exponential, the sums over n keys, the products: (n + 64) 2^-23 A.
    """
    k_codes, k_scale, v_codes, v_scale = cache
    n_pages, H, page, dh = k_codes.shape
    T, D = q.shape
    hq = D // dh
    out, tol = np.zeros((T, D)), np.zeros((T, D))
    q = q.astype(np.float64).reshape(T, hq, dh)
    q = hadamard_rows(q) if rotate else q
    for b in range(len(kv_len)):
        t0, t1 = int(cu[b]), int(cu[b + 1])
        n = int(kv_len[b])
        if t1 <= t0 or n <= 0:
            continue
        ids = table[b, np.arange(n) // page]
        ok = (ids >= 0) & (ids < n_pages)
        ids, at = np.where(ok, ids, 0), np.arange(n) % page
        for h in range(H):
            K = k_codes[ids, h, at].astype(np.float64) * np.where(ok, k_scale[ids, h], 0)[:, None]
            s_v = np.where(ok, v_scale[ids, h], 0).astype(np.float64)
            V = v_codes[ids, h, at].astype(np.float64) * s_v[:, None]
            for g in range(hq // H):
                c = h * (hq // H) + g
                s = q[t0:t1, c] @ K.T * scale
                S = np.abs(q[t0:t1, c]) @ np.abs(K).T * abs(scale)
                keep = ok & (np.arange(n)[None] <= (n - (t1 - t0) + np.arange(t1 - t0))[:, None])
                s = np.where(keep, s, -np.inf)
                m = s.max(1, keepdims=True)
                p = np.where(keep, np.exp(s - np.where(np.isfinite(m), m, 0)), 0)
                l = p.sum(1, keepdims=True)
                p = p / np.where(l > 0, l, 1)
                o, A = p @ V, p @ np.abs(V)
                e = np.where(keep, S, 0).max(1, keepdims=True) * (
                    (dh + 8) * 2.0 ** -24 + (2.0 ** -11 if q_rounded else 0))
                cols = slice(c * dh, (c + 1) * dh)
                out[t0:t1, cols] = o
                low = n * 2.0 ** -32 * 127 * np.where(keep, s_v[None], 0).max(1, keepdims=True)
                tol[t0:t1, cols] = (2.0 ** -8 * np.abs(o) + low
                                    + A * (2.0 ** -11 + np.expm1(2 * e) + (n + 64) * 2.0 ** -23))
    return out, tol
