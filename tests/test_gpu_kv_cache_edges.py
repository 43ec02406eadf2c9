"""The quantized KV cache on the GPU where its operators meet each other's edges
(needs an MI355X): pages of very unequal scales, lengths that a wave reads to
its last lane, requests that are refused and go on later. Against the float64
oracle, as in test_gpu_kv_cache.py."""
import numpy as np
import pytest

import workloads as W
from gpu_util import dev, host, say, torch
from oracle import kv_cache as K
from test_gpu_kv_cache import (FWHT, _attn_case, _cache, _check_attention, _i32, _kv_rows, _plan_case,
                               _run_attention, _same_cache, rw)  # noqa: F401 (rw: fixture)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- kv_attention: scales of the values
@pytest.mark.parametrize("up", [40, 100])
@pytest.mark.parametrize("ctx,new,group,dh,page", [
    ([0], [90], 1, 64, 16), ([100, 3], [130, 40], 2, 128, 16), ([37], [150], 1, 256, 32),   # by tiles
    ([3000], [100], 1, 64, 16),                                                               # in parts
    ([30, 13, 61], [9, 5, 4], 1, 64, 16), ([500, 14], [12, 12], 4, 128, 16),                 # by splits
    ([45], [6], 5, 256, 16), ([1270, 27], [3, 25], 1, 128, 16)])
def test_attention_later_scales(rw, ctx, new, group, dh, page, up):
    """A page of values 2^40 or 2^100 times as large leaves the rows alone that end
    before it, whatever tile they share with it."""
    say(f"kv_attention later scales ctx={ctx} new={new} group={group} dh={dh} page={page} up={up}")
    rng = np.random.default_rng(up + dh)
    cache, table, cu, kv_len, q, qg = _attn_case(rng, ctx, new, 1, group, dh, page)
    for b, n in enumerate(kv_len):
        cache[3][table[b, (n - 1) // page], 0] *= np.float32(2.0) ** up
    want, tol = K.kv_attention(q, cache, table, cu, kv_len, dh ** -0.5)
    got = _run_attention(rw, cache, table, cu, kv_len, qg, max(new), int(kv_len.max()), dh)
    _check_attention(got, want, tol)
    for b, n in enumerate(kv_len):                       # such rows exist, and are not zeros
        early = (n - 1) // page * page - ctx[b]
        if early > 0:
            assert np.abs(want[cu[b]:cu[b] + early]).max() > 0


@pytest.mark.parametrize("new", [[7, 12], [90, 40]])
def test_infinite_value_in_a_later_page(rw, new):
    """An infinity among a step's values fills its own page and head: the rows
    before that page keep their outputs."""
    say(f"infinite value new={new}")
    t = torch()
    rng = np.random.default_rng(6)
    H, page, dh, B = 2, 16, 64, 2
    ctx0 = [44, 13]
    width = 10
    want_cache = (np.zeros((B * width, H, page, dh), np.int8), np.zeros((B * width, H), np.float32),
                  np.zeros((B * width, H, page, dh), np.int8), np.zeros((B * width, H), np.float32))
    cache = rw.KvCache(*(dev(a) for a in want_cache))
    table = rng.permutation(B * width).reshape(B, width)
    ctx = np.zeros(B, int)
    for step in (ctx0, new):
        cu = np.concatenate([[0], np.cumsum(step)])
        pos = np.concatenate([np.arange(c, c + n) for c, n in zip(ctx, step)])
        slot = (table[np.repeat(np.arange(B), step), pos // page] * page + pos % page).astype(np.int64)
        (k, kg), (v, vg) = (_kv_rows(rng, len(slot), H * dh, "bf16") for _ in range(2))
        if step is new:
            for b in range(B):
                v[cu[b + 1] - 1, 5] = np.inf
                vg[cu[b + 1] - 1, 5] = 0x7F80
        K.kv_append(k, v, want_cache, cu, slot)
        rw.kv_append(dev(kg), dev(vg), cache, _i32(cu), dev(slot))
        ctx += np.array(step)
    t.cuda.synchronize()
    _same_cache(cache, want_cache)
    q, qg = _kv_rows(rng, sum(new), 2 * H * dh, "bf16")
    want, tol = K.kv_attention(q, want_cache, table, cu, ctx, 0.125)
    out = host(rw.kv_attention(dev(qg), cache, _i32(table), _i32(cu), _i32(ctx), max(new), int(ctx.max())))
    early = np.concatenate([np.arange(cu[b], cu[b + 1])[np.arange(ctx[b] - new[b], ctx[b]) <
                                                        (ctx[b] - 1) // page * page] for b in range(B)])
    assert len(early) > 4
    _check_attention(out[early], want[early], tol[early])


@pytest.mark.parametrize("ctx,new,group,dh", [
    ([300, 40], [1, 1], 4, 64), ([200], [10], 3, 128), ([9000, 300], [1, 1], 8, 64),
    ([3000, 90], [6, 6], 2, 256), ([60], [90], 1, 64), ([5000, 30], [70, 90], 1, 128), ([2500], [80], 1, 256)])
def test_attention_large_values(rw, ctx, new, group, dh):
    """Values so large that the sum over a row's keys would pass fp32's range,
    where their average does not; in one part and in several."""
    say(f"kv_attention large values ctx={ctx} new={new} group={group} dh={dh}")
    rng = np.random.default_rng(dh + group)
    cache, table, cu, kv_len, q, qg = _attn_case(rng, ctx, new, 1, group, dh, 16, q_scale=0.2)
    cache[2][:] = np.abs(cache[2])
    cache[3][:] = np.where(np.isnan(cache[3]), cache[3], np.float32(2.0) ** 119)
    want, tol = K.kv_attention(q, cache, table, cu, kv_len, dh ** -0.5)
    assert 2.0 ** 120 < want.min() and want.max() * 2 < np.finfo(np.float32).max
    for bound in (int(kv_len.max()), 20000):
        got = _run_attention(rw, cache, table, cu, kv_len, qg, max(new), bound, dh)
        _check_attention(got, want, tol)


# ---------------------------------------------------------------- requests that are not served
@pytest.mark.parametrize("captured", [False, True])
def test_refused_request_goes_on(rw, captured):
    """The pool runs out in the middle of a loop that feeds its own lengths back: a
    request that is not served keeps its tokens and pages, and goes on with its
    whole context once another has ended; no page is lost."""
    say(f"refused request goes on captured={captured}")
    t = torch()
    B, H, group, dh, page, n_pages, width = 3, 2, 2, 64, 16, 9, 7
    rng = np.random.default_rng(8)
    table, free, n_free = np.full((B, width), -1, np.int32), rng.permutation(n_pages).astype(np.int32), n_pages
    want_cache = [np.zeros(s, d) for s, d in (((n_pages, H, page, dh), np.int8), ((n_pages, H), np.float32)) * 2]
    cache = rw.kv_cache(n_pages, H, page, dh)
    T, D = 136, H * dh
    ctx = np.zeros(B, np.int32)
    s = {"ctx": _i32(ctx), "new": _i32(ctx), "table": dev(table), "free": dev(free), "n": _i32([n_free]),
         "x": t.zeros((T, (group + 2) * D), dtype=t.bfloat16, device="cuda"),
         "out": t.zeros((T, group * D), dtype=t.bfloat16, device="cuda"), "plan": None, "next": _i32(ctx)}
    need = rw.kv_attention_workspace_size(T, B, group * H, H, dh, 64, 112)
    ws = t.empty((max(need, 256),), dtype=t.uint8, device="cuda")

    def step():
        p = s["plan"] = rw.kv_plan(s["ctx"], s["new"], s["table"], s["free"], s["n"], T, page, out=s["plan"],
                                   ctx_next=s["next"])
        rw.kv_append(s["x"][:, -2 * D:-D], s["x"][:, -D:], cache, p.cu_new, p.slot)
        rw.kv_attention(s["x"][:, :-2 * D], cache, s["table"], p.cu_new, p.kv_len, 64, 112, out=s["out"],
                        workspace=ws)
        s["ctx"].copy_(s["next"])
        s["n"].copy_(p.n_free)
    step()                                               # no tokens: nothing changes; allocates the plan
    t.cuda.synchronize()
    graph = None
    if captured:
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph):
            step()
    refused = 0
    # 9 pages: 3 + 3 + 3; the second and third want a fourth and wait until the first ends
    for new in ([40, 48, 40], [1, 1, 1], [1, 9, 20], [0, 5, 2], [-1, 0, 0], [0, 9, 20], [0, 1, 1], [3, 0, -1]):
        x, bits = _kv_rows(rng, T, (group + 2) * D, "bf16")
        p = K.kv_plan(ctx, np.array(new), table, free, n_free, T, page)
        K.kv_append(x[:, -2 * D:-D], x[:, -D:], want_cache, p["cu_new"], p["slot"])
        out, tol = K.kv_attention(x[:, :-2 * D], want_cache, p["page_table"], p["cu_new"], p["kv_len"], 0.125)
        s["new"].copy_(_i32(new))
        s["x"].copy_(dev(bits))
        graph.replay() if captured else step()
        t.cuda.synchronize()
        for name in ("cu_new", "kv_len", "slot", "pos", "status", "n_free"):
            assert np.array_equal(host(getattr(s["plan"], name)), p[name]), (new, name)
        ctx = K.kv_ctx_next(ctx, p)
        assert np.array_equal(host(s["next"]), ctx)
        table, free, n_free = p["page_table"], p["free_pages"], int(p["n_free"][0])
        assert np.array_equal(host(s["table"]), table) and np.array_equal(host(s["free"]), free)
        _same_cache(rw.KvCache(*cache), want_cache)
        live = int(p["cu_new"][-1])
        if live:
            _check_attention(host(s["out"])[:live], out[:live], tol[:live])
        held = sum(-(-int(c) // page) for c in ctx)      # every page is a request's or free
        assert held + n_free == n_pages
        kept = np.concatenate([table[b, :-(-int(c) // page)] for b, c in enumerate(ctx)] + [free[:n_free]])
        assert sorted(kept.tolist()) == list(range(n_pages))
        refused += int((p["status"] == 1).sum())
    assert refused >= 4 and ctx.tolist() == [3, 58, 0]


def test_plan_most_rows(rw):
    """The most rows that a call takes, 2^30 - 1, and one token more: the request
    that it belongs to is refused, as with any other number of rows."""
    say("kv_plan with 2^30 - 1 rows")
    t = torch()
    T, page, half = 2 ** 30 - 1, 256, 2 ** 29
    pages = half // page
    for last, status in ((half - 1, 0), (half, 2)):
        table = t.full((2, pages), -1, dtype=t.int32, device="cuda")
        free = t.arange(2 * pages, dtype=t.int32, device="cuda")
        after = _i32([-1, -1])
        p = rw.kv_plan(_i32([0, 0]), _i32([half, last]), table, free, _i32([2 * pages]), T, page, ctx_next=after)
        t.cuda.synchronize()
        assert host(p.status).tolist() == [0, status] and host(p.cu_new).tolist() == [0, half, T]
        assert host(p.kv_len).tolist() == host(after).tolist() == [half, 0 if status else last]
        at = [0, 1, half - 1, half, half + 5, T - 1]
        want = [i if i < half else -1 if status else i - half for i in at]
        assert p.pos[at].tolist() == want
        top = 2 * pages - 1                              # pages from the top of the stack down
        assert p.slot[at].tolist() == [-1 if q < 0 else (top - i // page) * page + q % page for i, q in zip(at, want)]
        assert int(p.n_free) == (pages if status else 0)
        del p


def test_attention_join_of_many_rows(rw):
    """A batch of 2^21 rows and 32 heads whose last request is long enough for the
    tile kernel's parts: the join counts 2^26 rows and heads."""
    say("kv_attention join of 2^26 rows and heads")
    t = torch()
    T, heads, dh, page, n_pages, n, new, bound = 2 ** 21, 32, 64, 256, 40, 800000, 3, 2 ** 21
    rng = np.random.default_rng(22)
    cache, _, _, _, q, qg = _attn_case(rng, [n_pages * page - new], [new], 1, heads, dh, page)
    ids = np.argsort(np.isnan(cache[1][:, 0]))[:n_pages]     # the pages that hold something, again and again
    table = np.stack([np.zeros(-(-n // page), int), np.resize(ids, -(-n // page))])
    cu, kv_len = np.array([0, T - new, T]), np.array([0, n])
    need = rw.kv_attention_workspace_size(T, 2, heads, 1, dh, new, bound)
    assert need >= 2 * T * heads * (dh + 2) * 4              # parts of the tile kernel
    x = t.empty((T, heads * dh), dtype=t.bfloat16, device="cuda")
    x[-new:] = dev(qg)
    out = t.empty_like(x)
    out[-new - 1] = 7.0
    rw.kv_attention(x, rw.KvCache(*(dev(a) for a in cache)), _i32(table), _i32(cu), _i32(kv_len), new, bound,
                    out=out)
    t.cuda.synchronize()
    want, tol = K.kv_attention(q, cache, table[1:], [0, new], kv_len[1:], 0.125)
    _check_attention(host(out[-new:]), want, tol)
    assert not bool(out[:new].any()) and bool((out[-new - 1] == 7.0).all())


# ---------------------------------------------------------------- kv_attention: long parts
@pytest.mark.parametrize("H,group,dh,new,ctx,bound", [
    (8, 4, 64, 1, [130899], 131072),                         # parts of 4096 keys: 32 tiles a wave
    (8, 2, 128, 1, [130047], 131072),
    (32, 4, 64, 1, [4999, 300, 2047, 2048, 4095, 4096, 4500, 16, 3000, 2049, 1, 4998, 2300, 4200, 1000, 4400], 5000),
    (32, 2, 64, 1, [4095, 4000, 17, 2100, 4090, 1, 3500, 3200, 4094, 1025, 2050, 500, 4033, 1024, 3000, 2000], 4096),
    (64, 4, 64, 7, [4400, 2000, 90, 4100], 4500), (32, 3, 128, 9, [4000, 4060, 5, 2500, 3700, 900, 4071, 1500], 4096)])
def test_attention_long_parts(rw, H, group, dh, new, ctx, bound):
    """Parts of up to 4096 keys, whose waves look 64 blocks of keys up at once; with
    pages that are not there at the last block of a wave. Three heads against the
    oracle."""
    say(f"kv_attention long parts H={H} group={group} dh={dh} new={new} bound={bound}")
    page, B = 16, len(ctx)
    rng = np.random.default_rng(H + dh + new)
    kv_len = np.array(ctx) + new
    used = -(-kv_len // page)
    n_pages = int(used.sum())
    table = np.full((B, int(used.max())), -1)
    first = np.concatenate([[0], np.cumsum(used)])
    perm = rng.permutation(n_pages)
    for b in range(B):
        table[b, :used[b]] = perm[first[b]:first[b + 1]]
    for b in range(B):                                       # blocks 31, 63, 64, 127, ... are missing in turn
        gone = np.arange(31 + 32 * (b % 3), used[b] - 1, 97 if b % 2 else 64)
        table[b, gone] = [-1, n_pages, 2 ** 31 - 1][b % 3]
    heads = [0, H // 2 - 1, H - 1]
    cache, sample = [], []
    for i in range(4):
        a = rng.integers(-127, 128, (n_pages, H, page, dh), np.int8) if i % 2 == 0 else \
            (0.01 + 0.02 * rng.random((n_pages, H), np.float32))
        cache.append(dev(a))
        sample.append(np.ascontiguousarray(a[:, heads]))
    cu = np.arange(B + 1) * new
    q, qg = _kv_rows(rng, B * new, H * group * dh, "bf16")
    out = host(rw.kv_attention(dev(qg), rw.KvCache(*cache), _i32(table), _i32(cu), _i32(kv_len), new, bound,
                               scale=0.02))
    cols = np.concatenate([np.arange(h * group * dh, (h + 1) * group * dh) for h in heads])
    want, tol = K.kv_attention(np.ascontiguousarray(q[:, cols]), sample, table, cu, kv_len, 0.02)
    _check_attention(out[:, cols], want, tol)
    got = W.bf16_bits_to_f32(out)
    assert np.isfinite(got).all() and (np.abs(got).max(1) > 0).all()


# ---------------------------------------------------------------- kv_append: values that are not finite
@pytest.mark.parametrize("together", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_append_not_finite_among_others(rw, dt, together):
    """A NaN or an infinity between ordinary tokens, appended with them or one by one."""
    say(f"kv_append not finite together={together} {dt}")
    H, page, dh, n = 2, 16, 64, 18
    rng = np.random.default_rng(23)
    x, bits = _kv_rows(rng, n, H * dh, dt)
    y, ybits = _kv_rows(rng, n, H * dh, dt)
    x[3, 5], y[7, 70] = np.nan, -np.inf
    bits[3, 5], ybits[7, 70] = (0x7FC0, 0xFF80) if dt == "bf16" else (np.nan, -np.inf)
    want, cache = _cache(rw, 2, H, page, dh)
    slot = np.arange(n)
    step = n if together else 1
    for t in range(0, n, step):
        K.kv_append(x[t:t + step], y[t:t + step], want, [0, step], slot[t:t + step])
        rw.kv_append(dev(bits[t:t + step]), dev(ybits[t:t + step]), cache, _i32([0, step]), dev(slot[t:t + step]))
    torch().cuda.synchronize()
    _same_cache(cache, want)
    assert want[1].max() < 100 and want[3][0, 1] > 2e36 and want[3][0, 0] < 100 and want[3][1].max() < 100
    kept = want[2][0, 1].copy()                              # the infinity's page and head hold it alone
    kept[7, 6] = 0
    assert want[2][0, 1, 7, 6] == -127 and not kept.any()


# ---------------------------------------------------------------- kv_attention: far scores of rounded queries
@pytest.mark.parametrize("q_scale", [6.0, 16.0])
@pytest.mark.parametrize("dt,rotate", [("bf16", True), ("f32", False), ("f32", True)])
@pytest.mark.parametrize("ctx,new,group,dh", [
    ([700, 33], [1, 1], 4, 64), ([300], [6], 4, 128), ([200], [5], 4, 256), ([200, 5], [90, 70], 1, 128),
    ([2500], [80], 1, 64)])
def test_attention_far_scores(rw, ctx, new, group, dh, dt, rotate, q_scale):
    """Transformed and fp32 queries, which are rounded to fp16, where the scores are
    far apart and few keys have the weight."""
    say(f"kv_attention far scores {ctx} {new} group={group} dh={dh} {dt} rotate={rotate} {q_scale}")
    rng = np.random.default_rng(24 + dh)
    cache, table, cu, kv_len, q, qg = _attn_case(rng, ctx, new, 2, group, dh, 32, dt, q_scale)
    want, tol = K.kv_attention(q, cache, table, cu, kv_len, dh ** -0.5, rotate, True)
    got = _run_attention(rw, cache, table, cu, kv_len, qg, max(new), int(kv_len.max()), dh, rotate)
    say(f"  worst error {_check_attention(got, want, tol):.2f} of the bound")


@pytest.mark.parametrize("B,page,max_ctx,max_new,ended,spare", [
    (1, 16, 40, 3, 0, 0), (20, 16, 60, 30, 2, -9), (300, 16, 60, 30, 9, -40), (257, 64, 900, 3, 50, 5)])
def test_plan_next_lengths(rw, B, page, max_ctx, max_new, ended, spare):
    """The next step's lengths beside a plan that is the same with and without them;
    requests served, ended, without pages and with lengths out of range."""
    say(f"kv_plan ctx_next B={B} spare={spare}")
    rng = np.random.default_rng(B)
    ctx, new, table, free, n_free = _plan_case(rng, B, page, max_ctx, max_new, ended, spare=max(spare, 0))
    n_free = max(0, n_free + min(spare, 0))
    if B > 20:
        ctx[7], new[8], ctx[9] = -3, -2, table.shape[1] * page + 1
    T = int(np.maximum(new, 0).sum()) - (5 if B == 257 else 0)
    want = K.kv_plan(ctx, new, table, free, n_free, T, page)
    args = (_i32(ctx), _i32(new), dev(table), dev(free), _i32([n_free]))
    after = _i32(np.full(B, -9))
    plan = rw.kv_plan(*args, T, page, ctx_next=after)
    torch().cuda.synchronize()
    assert np.array_equal(host(after), K.kv_ctx_next(ctx, want))
    got = dict(plan._asdict(), page_table=args[2], free_pages=args[3])
    for name, w in want.items():
        assert np.array_equal(host(got[name]), w), name
    for bad in (after[:-1], after.long(), after.cpu()):
        with pytest.raises(ValueError):
            rw.kv_plan(*args, T, page, ctx_next=bad)
    with pytest.raises(rw.Rw4Error):
        rw.kv_plan(*args, T, page, ctx_next=args[0])
