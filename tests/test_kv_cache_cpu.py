"""The quantized KV cache on the CPU: the entry points refuse invalid arguments
before any device work, and the oracle holds on cases worked out by hand."""
import ctypes

import numpy as np
import pytest

import rotation_w4a4_quantized_amd as rw
from oracle import kv_cache as K

P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(12)]
NUL = None
ODD = ctypes.c_void_p(0x10004)     # 4-byte aligned only
OFF = ctypes.c_void_p(0x10002)     # not even that
INV, UNS, MIS, WSE = -1, -2, -3, -4


def _plan(ctx=P[0], new=P[1], B=4, table=P[2], width=8, page=64, free=P[3], cap=100, n=P[4],
          n_out=P[5], cu=P[6], kv=P[7], slot=P[8], pos=P[9], status=P[10], T=4):
    return rw.lib().kv_plan(ctx, new, B, table, width, page, free, cap, n, n_out, cu, kv, slot, pos,
                            status, T, NUL)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=0), INV), (dict(B=4097), UNS), (dict(T=-1), INV), (dict(width=0), INV),
    (dict(cap=0), INV), (dict(page=48), UNS), (dict(page=8), UNS), (dict(page=512), UNS),
    (dict(T=1 << 30), UNS), (dict(cap=1 << 30), UNS), (dict(width=1 << 25, page=64), UNS),
    (dict(B=4096, width=1 << 18), UNS),
    (dict(ctx=NUL), INV), (dict(new=NUL), INV), (dict(table=NUL), INV), (dict(free=NUL), INV),
    (dict(n=NUL), INV), (dict(n_out=NUL), INV), (dict(cu=NUL), INV), (dict(kv=NUL), INV),
    (dict(slot=NUL), INV), (dict(pos=NUL), INV), (dict(status=NUL), INV),
    (dict(n_out=P[4]), INV), (dict(kv=P[0]), INV), (dict(cu=P[1]), INV), (dict(status=P[1]), INV),
    (dict(ctx=OFF), MIS), (dict(table=OFF), MIS), (dict(slot=ODD), MIS), (dict(pos=OFF), MIS),
])
def test_plan_validation(kw, expect):
    assert _plan(**kw) == expect


def _append(k=P[0], v=P[1], dt=0, ldk=512, ldv=512, T=4, B=2, flags=0, cu=P[2], slot=P[3],
            kc=P[4], ks=P[5], vc=P[6], vs=P[7], n_pages=10, H=4, page=64, dh=128):
    return rw.lib().kv_append(k, v, dt, ldk, ldv, T, B, flags, cu, slot, kc, ks, vc, vs, n_pages,
                              H, page, dh, NUL)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), INV), (dict(B=-1), INV), (dict(dt=2), INV), (dict(flags=1), INV),
    (dict(flags=2 | 4), INV), (dict(H=0), INV), (dict(n_pages=-1), INV), (dict(page=24), UNS),
    (dict(dh=96), UNS), (dict(dh=32), UNS), (dict(H=65536, ldk=1 << 24, ldv=1 << 24), UNS),
    (dict(T=1 << 30), UNS), (dict(B=1 << 30), UNS), (dict(n_pages=1 << 30), UNS),
    (dict(B=1 << 24, H=65535, ldk=1 << 24, ldv=1 << 24), UNS),
    (dict(T=1 << 27, page=256, k=NUL), UNS), (dict(T=(1 << 27) - 512, page=256, k=NUL), INV),
    (dict(ldk=504), INV), (dict(ldv=516), INV), (dict(ldk=514, dt=1), INV),
    (dict(k=NUL), INV), (dict(v=NUL), INV), (dict(cu=NUL), INV), (dict(slot=NUL), INV),
    (dict(kc=NUL), INV), (dict(ks=NUL), INV), (dict(vc=NUL), INV), (dict(vs=NUL), INV),
    (dict(k=ODD), MIS), (dict(v=ODD), MIS), (dict(kc=ODD), MIS), (dict(vs=OFF), MIS),
    (dict(slot=ODD), MIS), (dict(cu=OFF), MIS),
    (dict(T=0, k=NUL, v=NUL, slot=NUL, kc=NUL), 0), (dict(B=0, cu=NUL), 0),
])
def test_append_validation(kw, expect):
    assert _append(**kw) == expect


def _attend(q=P[0], dt=0, ldq=1024, out=P[1], ldo=1024, T=4, B=2, Hq=8, scale=0.1, flags=0,
            cu=P[2], kv=P[3], table=P[4], width=16, kc=P[5], ks=P[6], vc=P[7], vs=P[8],
            n_pages=40, H=4, page=64, dh=128, max_new=4, max_kv=512, ws=P[9], nb=1 << 30):
    return rw.lib().kv_attention(q, dt, ldq, out, ldo, T, B, Hq, scale, flags, cu, kv, table, width,
                                 kc, ks, vc, vs, n_pages, H, page, dh, max_new, max_kv, ws, nb, NUL)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), INV), (dict(B=-1), INV), (dict(dt=2), INV), (dict(flags=1), INV),
    (dict(Hq=0), INV), (dict(Hq=6, H=4), INV), (dict(scale=float("nan")), INV),
    (dict(scale=float("inf")), INV), (dict(max_new=-1), INV), (dict(max_kv=-1), INV),
    (dict(width=0), INV), (dict(page=100), UNS), (dict(dh=192), UNS), (dict(B=65536), UNS),
    (dict(T=1 << 30), UNS), (dict(Hq=65536, ldq=1 << 24, ldo=1 << 24), UNS),
    (dict(width=1 << 25), UNS), (dict(max_kv=1 << 26), UNS), (dict(max_new=1 << 30), UNS),
    (dict(B=65535, H=129, Hq=129, ldq=1 << 16, ldo=1 << 16), UNS), (dict(n_pages=0), INV),
    (dict(n_pages=1 << 29, page=128), UNS),
    (dict(ldq=1016), INV), (dict(ldo=1016), INV), (dict(ldq=1028), INV), (dict(ldo=1028), INV),
    (dict(ldq=1026, dt=1), INV), (dict(q=NUL), INV), (dict(out=NUL), INV), (dict(cu=NUL), INV),
    (dict(kv=NUL), INV), (dict(table=NUL), INV), (dict(kc=NUL), INV), (dict(vs=NUL), INV),
    (dict(out=P[0]), INV), (dict(q=ODD), MIS), (dict(out=ODD), MIS), (dict(vc=ODD), MIS),
    (dict(ks=OFF), MIS), (dict(kv=OFF), MIS),
    (dict(T=0, q=NUL, out=NUL, ws=NUL), 0), (dict(B=0), 0), (dict(max_new=0), 0),
])
def test_attention_validation(kw, expect):
    assert _attend(**kw) == expect


def test_attention_workspace():
    size = rw.lib().kv_attention_workspace_size
    for bad in ((0, 1, 8, 8, 128, 1, 64), (1, 0, 8, 8, 128, 1, 64), (1, 1, 7, 2, 128, 1, 64),
                (1, 1, 8, 8, 96, 1, 64), (1, 1, 8, 0, 128, 1, 64), (-1, 1, 8, 8, 128, 1, 64),
                (1, 65536, 8, 8, 128, 1, 64), (1, 1, 8, 8, 128, 0, 64), (1, 1, 8, 8, 128, 1, 0)):
        assert size(*bad) == 0
    need = size(1, 1, 64, 8, 128, 1, 131072)
    if need:                                        # a long cache is split and joined
        kw = dict(T=1, B=1, Hq=64, H=8, ldq=8192, ldo=8192, max_new=1, max_kv=131072)
        assert _attend(**kw, ws=NUL) == WSE and _attend(**kw, nb=need - 1) == WSE
        assert _attend(**kw, ws=ODD) == WSE


# ---------------------------------------------------------------- the oracle
def test_oracle_plan_by_hand():
    """Pages of 16: request 0 grows into one new page, request 1 ends, request 2
    starts with 20 tokens."""
    table = np.full((3, 4), -1, np.int32)
    table[0, :1], table[1, :2] = 5, (7, 8)
    free = np.array([1, 2, -9, -9, -9], np.int32)
    o = K.kv_plan(np.array([16, 17, 0]), np.array([1, -1, 20]), table, free, 2, 23, 16)
    assert o["free_pages"].tolist() == [1, 2, 7, 8, -9]      # 7 and 8 given back
    assert o["page_table"].tolist() == [[5, 8, -1, -1], [7, 8, -1, -1], [7, 2, -1, -1]]
    assert o["slot"].tolist() == [8 * 16] + [7 * 16 + i for i in range(16)] + \
        [2 * 16 + i for i in range(4)] + [-1, -1]
    assert o["pos"].tolist() == [16] + list(range(20)) + [-1, -1]
    assert o["kv_len"].tolist() == [17, 0, 20] and o["n_free"].tolist() == [1]
    assert o["cu_new"].tolist() == [0, 1, 1, 21] and o["status"].tolist() == [0, 0, 0]


def test_oracle_append_by_hand():
    """absmax 127 gives step 1; a later row of absmax 254 doubles it and halves
    the older codes (half to even)."""
    cache = (np.full((2, 1, 16, 64), 99, np.int8), np.full((2, 1), 9, np.float32),
             np.full((2, 1, 16, 64), 99, np.int8), np.full((2, 1), 9, np.float32))
    x = np.zeros((1, 64), np.float32)
    x[0, :5] = 127, -127, 1, 2.5, 3
    K.kv_append(x, x, cache, [0, 1], [16])                    # opens page 1: its old scale is void
    assert cache[1].tolist() == [[9], [1]]
    assert cache[0][1, 0, 0, :6].tolist() == [127, -127, 1, 2, 3, 0]
    K.kv_append(2 * x, x, cache, [0, 1], [17])
    assert cache[1].tolist() == [[9], [2]] and cache[3].tolist() == [[9], [1]]
    assert cache[0][1, 0, 0, :6].tolist() == [64, -64, 0, 1, 2, 0]
    assert cache[0][1, 0, 1, :6].tolist() == [127, -127, 1, 2, 3, 0]
    assert (cache[0][0] == 99).all() and (cache[0][1, 0, 2:] == 99).all()


def test_oracle_attention_by_hand():
    """Equal scores average the values; one key gives its value; a query before
    the first key gives 0."""
    cache = (np.zeros((1, 1, 16, 64), np.int8), np.ones((1, 1), np.float32),
             np.zeros((1, 1, 16, 64), np.int8), np.full((1, 1), 0.5, np.float32))
    cache[2][0, 0, :3, 0] = 2, 4, 12
    q = np.ones((3, 64))
    table = np.zeros((1, 1), np.int32)
    out, tol = K.kv_attention(q, cache, table, [0, 3], [3], 1.0)
    assert out[:, 0].tolist() == [1, 1.5, 3] and (out[:, 1:] == 0).all() and (tol[:, 0] > 0).all()
    out, _ = K.kv_attention(q, cache, table, [0, 3], [2], 1.0)
    assert out[:, 0].tolist() == [0, 1, 1.5]


def test_oracle_transform_is_orthogonal():
    x = np.random.default_rng(0).standard_normal((3, 128))
    y = K.hadamard_rows(x)
    assert np.allclose(K.hadamard_rows(y), x) and np.allclose((x * x).sum(1), (y * y).sum(1))
    assert np.allclose(K.hadamard_rows(np.array([[20.0, 0, 0, 0]])), 10)


def test_workspace_of_a_mixed_batch():
    """One generated token at a long context beside a prompt of 4096: the parts of
    the long context are kept for the few rows that have them."""
    alone = rw.kv_attention_workspace_size(4, 4, 32, 8, 128, 1, 1 << 20)
    both = rw.kv_attention_workspace_size(4099, 4, 32, 8, 128, 4096, 1 << 20)
    prompt = rw.kv_attention_workspace_size(4099, 1, 32, 8, 128, 4099, 1 << 20)
    assert 0 < alone <= both <= prompt + 16 * alone


def _plan_next(ctx=P[0], new=P[1], after=P[11], T=4):
    return rw.lib().kv_plan_next(ctx, new, 4, P[2], 8, 64, P[3], 100, P[4], P[5], P[6], P[7], P[8], P[9], P[10], T,
                                 after, NUL)


@pytest.mark.parametrize("kw,expect", [
    (dict(after=NUL), INV), (dict(after=P[0]), INV), (dict(after=P[1]), INV), (dict(after=OFF), MIS),
    (dict(ctx=NUL), INV), (dict(T=-1), INV), (dict(T=1 << 30), UNS)])
def test_plan_next_validation(kw, expect):
    assert _plan_next(**kw) == expect


def test_oracle_plan_refused_by_hand():
    """One free page for two requests: the first takes it, the second keeps its 16
    tokens and page 7; lengths out of range stay as they are."""
    table = np.full((4, 2), -1, np.int32)
    table[0, 0], table[1, 0], table[3, 0] = 5, 7, 8
    o = K.kv_plan(np.array([16, 16, 99, 4]), np.array([1, 1, 1, -1]), table[:, :], np.array([3, -9, -9]), 1, 9, 16)
    assert o["status"].tolist() == [0, 0, 2, 0]              # page 8 comes back first
    o = K.kv_plan(np.array([16, 16, 99, 4]), np.array([1, 1, 1, 0]), table, np.array([3, -9, -9]), 1, 9, 16)
    assert o["status"].tolist() == [0, 1, 2, 0] and o["kv_len"].tolist() == [17, 0, 0, 4]
    assert K.kv_ctx_next([16, 16, 99, 4], o).tolist() == [17, 16, 99, 4] and o["n_free"].tolist() == [0]
    assert o["page_table"].tolist() == [[5, 3], [7, -1], [-1, -1], [8, -1]]


@pytest.mark.parametrize("args", [
    (1, 1, 64, 8, 128, 1, 131072), (1, 1, 8, 8, 64, 1, 4096), (64, 64, 32, 8, 128, 1, 16384),
    (16, 16, 128, 32, 64, 1, 5000), (70, 1, 2, 1, 256, 70, 2600), (512, 1, 32, 8, 128, 512, 8704)])
def test_attention_workspace_of_split_keys(args):
    """Calls whose keys are split need a workspace, for two parts at least of every
    row and head, and refuse a smaller one."""
    T, B, Hq, H, dh, max_new, max_kv = args
    need = rw.lib().kv_attention_workspace_size(*args)
    assert need >= 2 * T * Hq * (dh + 2) * 4
    kw = dict(T=T, B=B, Hq=Hq, H=H, dh=dh, ldq=Hq * dh, ldo=Hq * dh, max_new=max_new, max_kv=max_kv)
    assert _attend(**kw, ws=NUL) == WSE and _attend(**kw, nb=need - 1) == WSE and _attend(**kw, ws=ODD) == WSE


def test_oracle_append_not_finite_by_hand():
    """A NaN is a 0 in its place and nothing else; an infinity takes the scale of its
    page and head to FLT_MAX / 127, where older and later values have code 0; the
    other head and the next page keep theirs."""
    def empty():
        return tuple(np.zeros(s, d) for s, d in (((2, 2, 16, 64), np.int8), ((2, 2), np.float32)) * 2)
    x = np.ones((18, 128), np.float32)
    x[:, [0, 64]] = 127
    slots = np.arange(18)
    c = empty()
    bad = x.copy()
    bad[3, 5] = np.nan
    K.kv_append(bad, x, c, [0, 18], slots)
    assert c[1].tolist() == [[1, 1], [1, 1]] and c[0][0, 0, 3, 4:7].tolist() == [1, 0, 1]
    assert (c[0][0, :, :3, 0] == 127).all() and (c[0][0, 1] == c[2][0, 1]).all()
    c = empty()
    bad = x.copy()
    bad[3, 5] = -np.inf
    for t in range(18):                                      # token by token
        K.kv_append(bad[t:t + 1], x[t:t + 1], c, [0, 1], slots[t:t + 1])
    top = np.finfo(np.float32).max / np.float32(127)
    assert c[1].tolist() == [[top, 1], [1, 1]] and c[3].tolist() == [[1, 1], [1, 1]]
    want = np.zeros((16, 64))
    want[3, 5] = -127
    assert (c[0][0, 0] == want).all() and (c[0][0, 1, :, 0] == 127).all() and (c[0][1, 0, :2, 0] == 127).all()


@pytest.mark.parametrize("T,B,Hq,H,dh,max_new,max_kv", [
    (3000, 2, 32, 8, 128, 1500, 1500), (3800, 2, 32, 8, 128, 1900, 1900), (3600, 3, 32, 8, 128, 1200, 1200),
    (3000, 2, 32, 32, 128, 1500, 1500), (3000, 2, 32, 8, 64, 1500, 1500), (2408, 3, 32, 8, 128, 1099, 1099),
    (3584, 7, 32, 8, 128, 512, 8512)])
def test_prompts_that_fill_the_card_take_one_part(T, B, Hq, H, dh, max_new, max_kv):
    """Prompts with 256 to 511 workgroups, whose keys in parts take 15 to 60% longer
    than in one: no parts, no workspace, as with fewer and more workgroups."""
    assert rw.kv_attention_workspace_size(T, B, Hq, H, dh, max_new, max_kv) == 0
