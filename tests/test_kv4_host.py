"""CPU checks of the 4-bit cache: the oracle's number format pinned by other means, and the refusals of
the entry points (checked before any device call)."""

import numpy as np
import pytest

import oracle.kv4 as K4
import oracle.kv8 as K8
from shared_prefix_kv_decode_gb300 import _binding as gb


def _ctx(n_q=8, n_kv=2, d=64, dtype=gb.DTYPE_BF16, max_batch=8, **kw):
    return gb.Context(n_layers=1, n_q=n_q, n_kv=n_kv, head_dim=d, dtype=dtype, n_slots=1000, hot_fraction=0.5,
                      max_batch=max_batch, host_only=True, **{"kv4": True, **kw})


def _status(call, *args):
    with pytest.raises(gb.GranikvError) as e:
        call(*args)
    return e.value.status


def test_codes_are_nearest_with_ties_to_even():
    grid = np.concatenate([K4.E2M1, [8.0]])
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(0, 9, 4000), rng.uniform(0, 0.6, 500), K4.E2M1, (K4.E2M1[:-1] + K4.E2M1[1:]) / 2, [5.0, 1e9, np.inf, 0.0]])
    codes = K4.e2m1_codes(x)
    for a, c in zip(x, codes):
        if a >= 6:
            assert c == 7
            continue
        dist = np.abs(K4.E2M1 - a)
        best = np.flatnonzero(dist == dist.min())
        assert c in best and (len(best) == 1 or c % 2 == 0)
    assert np.array_equal(K4.e2m1_codes(-x), codes | 8)
    assert (np.diff(grid) > 0).all()


@pytest.mark.parametrize("block", [1, K4.BLOCK])
def test_quantise_by_its_definition(block):
    """The exponent is the least that holds amax, a scale is within half a step of bmax / 6, and a value within
    half a step of what it stands for, or at the largest one below it (a scale may be rounded down)."""
    rng = np.random.default_rng(block)
    x = (rng.standard_normal((130, 3, 64)) * np.exp2(rng.uniform(-30, 30, (130, 1, 1)))).astype(np.float32)
    x[5] = 0.0
    x[7, 1] = 2.0 ** 11 * 1.3125  # exactly 2688: exponent 0
    x[8, 1] = np.nextafter(np.float32(2688), np.float32(1e9))
    codes, scale, e = K4.quantise(x, block)
    unit = np.ldexp(1.0, e.astype(int) - 127)
    amax = np.abs(x).max(axis=2).astype(np.float64)
    for t in range(0, 130, block):
        amax[t:t + block] = amax[t:t + block].max(axis=0)
    assert (amax <= 2688 * unit).all() and ((amax > 1344 * unit) | (e == 127 + K4.EXP_MIN)).all()
    if block == 1:
        assert e[7, 1] == 127 and e[8, 1] == 128
    b = K8.e4m3_values()[scale]
    y = np.abs(x).reshape(130, 3, 4, 16).max(axis=3) / (6 * unit[..., None])
    assert (np.abs(b - y) <= np.maximum(y * 2.0 ** -4, 2.0 ** -9)).all() and (b >= 2.0 ** -9).all()
    v = K4.values(codes, scale, e).reshape(130, 3, 4, 16)
    step = np.where(np.abs(v) >= 4 * (b * unit[..., None])[..., None], 2.0, np.where(np.abs(v) >= 2 * (b * unit[..., None])[..., None], 1.0, 0.5))
    off = np.abs(v - x.reshape(v.shape))
    one = (b * unit[..., None])[..., None]
    assert (off <= np.maximum(one * step / 2 * (1 + 1e-12), np.abs(x.reshape(v.shape)) - 6 * one)).all()
    assert np.array_equal(v.astype(np.float32).astype(np.float64), v)  # exact in fp32


def test_quantise_edges():
    x = np.zeros((2, 2, 32), dtype=np.float32)
    x[0, 0, :4] = [6.0, -3.0, np.inf, -0.0]
    x[0, 1, 0], x[0, 1, 20] = np.nan, 12.0
    x[1, 0] = 3e38
    x[1, 1] = 1e-40
    codes, scale, e = K4.quantise(x, 1)
    assert list(codes[0, 0, :4]) == [7, 13, 7, 8]
    assert scale[0, 1, 0] == 0x7F and scale[0, 1, 1] != 0x7F and np.isfinite(K4.values(codes, scale, e)[0, 1, 16:]).all()
    assert np.isnan(K4.values(codes, scale, e)[0, 1, :16]).all()
    assert e[1, 0] == 127 + K4.EXP_MAX and np.isfinite(K4.values(codes, scale, e)[1, 0].astype(np.float32)).all()
    assert e[1, 1] == 127 + K4.EXP_MIN and not (codes[1, 1] & 7).any() and (scale[1, 1] == 1).all()


@pytest.mark.parametrize("n_kv,d,want", [(8, 128, 592), (1, 32, 48), (3, 96, 192), (2, 64, 96), (5, 256, 736), (1, 128, 96)])
def test_row_bytes(granikv_lib, n_kv, d, want):
    assert gb.kv4_row_bytes(n_kv, d) == want == K4.row_bytes(n_kv, d)


def test_row_bytes_refusals(granikv_lib):
    assert _status(gb.kv4_row_bytes, 0, 64) == gb.ERR_INVALID
    for d in (0, 16, 31, 48, 288):
        assert _status(gb.kv4_row_bytes, 2, d) == gb.ERR_UNSUPPORTED
    assert gb.kv4_row_bytes(2 ** 24 // 145 - 1, 256) <= 2 ** 24
    for n_kv in (2 ** 24 // 145 + 1, 2 ** 30):
        assert _status(gb.kv4_row_bytes, n_kv, 256) == gb.ERR_UNSUPPORTED
        with pytest.raises(gb.GranikvError) as e:
            _ctx(n_q=n_kv, n_kv=n_kv, d=256)
        assert e.value.status == gb.ERR_UNSUPPORTED


def test_kv4_context_refusals(granikv_lib):
    with pytest.raises(ValueError):
        _ctx(kv8=True)
    with pytest.raises(gb.GranikvError) as e:
        _ctx(d=80)
    assert e.value.status == gb.ERR_UNSUPPORTED
    ctx = _ctx()
    sid, _ = ctx.hot_alloc(100)
    assert _status(ctx.hot_fill, 0, sid, 4096, 4096 + 8) == gb.ERR_INVALID
    assert _status(ctx.hot_fill, 0, sid, 4096, 4096) == gb.ERR_NO_DEVICE
    assert _status(ctx.cold_append, 0, 4098, 4096, 4096, 3) == gb.ERR_INVALID
    assert _status(ctx.cold_append, 0, 4096, 4096, 4096, 3) == gb.ERR_NO_DEVICE
    b = gb.Batch([sid], [3], 4096, 16, 4096)
    assert _status(ctx.decode_attention, 0, 4100, b, None, 4096, 4096, 4096, 1 << 20) == gb.ERR_INVALID
    assert _status(ctx.decode_attention, 0, 4096, b, None, 4104, 4096, 4096, 1 << 20) == gb.ERR_INVALID
    assert _status(ctx.decode_attention, 0, 4096, b, None, 4096, 4096, 4096, 1 << 20) == gb.ERR_NO_DEVICE
    assert _status(ctx.cold_weigh, 0, 4100, 4096, b, 4096) == gb.ERR_INVALID
    assert _status(ctx.cold_weigh, 0, 4096, 4096, b, 4096) == gb.ERR_NO_DEVICE


@pytest.mark.parametrize("kind", [{"kv4": True}, {"kv4": False, "kv8": True}, {"kv4": False}])
def test_read_refusals(granikv_lib, kind):
    ctx = _ctx(**kind)
    sid, _ = ctx.hot_alloc(100)
    assert _status(ctx.hot_read, 0, sid, 0, 100, 4096, 4096) == gb.ERR_NO_DEVICE
    assert _status(ctx.hot_read, 0, sid, 100, 0, None, None) == gb.ERR_NO_DEVICE
    for args in [(1, sid, 0, 5, 4096, 4096), (-1, sid, 0, 5, 4096, 4096), (0, sid + 1, 0, 5, 4096, 4096), (0, -1, 0, 5, 4096, 4096),
                 (0, sid, -1, 5, 4096, 4096), (0, sid, 0, -1, 4096, 4096), (0, sid, 96, 5, 4096, 4096), (0, sid, 0, 101, 4096, 4096),
                 (0, sid, 2 ** 31 - 1, 2 ** 31 - 1, 4096, 4096), (0, sid, 0, 5, None, 4096), (0, sid, 0, 5, 4096, None),
                 (0, sid, 0, 5, 4104, 4096), (0, sid, 0, 5, 4096, 4100)]:
        assert _status(ctx.hot_read, *args) == gb.ERR_INVALID, args
    assert _status(ctx.cold_read, 0, 4096, 5, 4096, 4096) == gb.ERR_NO_DEVICE
    for args in [(1, 4096, 5, 4096, 4096), (0, None, 5, 4096, 4096), (0, 4096, -1, 4096, 4096), (0, 4096, 5, None, 4096),
                 (0, 4096, 5, 4096, None), (0, 4096, 5, 4098, 4096), (0, 4096, 5, 4096, 4104)]:
        assert _status(ctx.cold_read, *args) == gb.ERR_INVALID, args
    ctx.hot_free(sid)
    assert _status(ctx.hot_read, 0, sid, 0, 1, 4096, 4096) == gb.ERR_INVALID


def test_kv4_dispatch_plans(granikv_lib):
    for d in (64, 128):
        ctx = _ctx(d=d)
        sid, _ = ctx.hot_alloc(300)
        plan = ctx.dispatch(gb.Batch([sid, -1, sid], [5, 40, 0], 4096, 64))
        (grp,) = plan.groups()
        assert grp["slab_id"] == sid and grp["n_requests"] == 2 and grp["L_p"] == 300
        assert ctx.workspace_size(plan) > 0


def test_dense_kernel_reads_ahead(granikv_lib):
    """One content ahead over the 4-bit cache, unless it is set; none where the others' split does not ask for it."""
    for kw, want in ((dict(kv4=True), 1), (dict(kv8=True), 0)):
        ctx = gb.Context(n_layers=1, n_q=32, n_kv=8, head_dim=128, dtype=gb.DTYPE_BF16, n_slots=4000, hot_fraction=0.5, host_only=True, **kw)
        sid, _ = ctx.hot_alloc(1000)
        batch = gb.Batch([sid, sid], [0, 0], 4096, 64)
        assert ctx.dispatch(batch).dense_l2_ahead() == want
        ctx.set_dense_l2_ahead(0)
        assert ctx.dispatch(batch).dense_l2_ahead() == 0


def _plan_case(rng):
    n_prefix = int(rng.choice([1, 1, 2, 5, 20]))
    B = int(rng.choice([1, 2, 7, 40, 200, 1000]))
    prefixes = [int(np.exp(rng.uniform(0, 11))) for _ in range(n_prefix)]
    top = np.exp(rng.uniform(0, 9))
    lens = [int(rng.uniform(0, 40000)) if rng.random() < 0.1 else int(rng.uniform(0, top)) for _ in range(B)]
    n_q, n_kv = [(8, 8), (32, 8), (40, 8), (64, 8), (16, 4), (8, 1), (6, 2), (24, 12), (32, 16)][int(rng.integers(9))]
    return prefixes, lens, n_q, n_kv


PLANS = [_plan_case(np.random.default_rng([4, s])) for s in range(40)] + [
    ([16384], [300] * 8, 32, 8), ([8192], [250], 32, 8), ([16384], [1] * 64, 32, 8), ([100000], [300000, 1], 32, 8),
    ([100], [200000, 3, 5, 7], 32, 8), ([16384], [100] * 4000, 32, 8), ([500], [0, 1, 2, 3] * 1000, 32, 8), ([64], [8192] * 16, 32, 8)]


@pytest.mark.parametrize("group", range(0, len(PLANS), 10))
@pytest.mark.parametrize("schedule", [(True, 0.0), (True, 0.5), (False, 0.0)])
@pytest.mark.parametrize("d", [128, 64])
def test_plans_cover_every_token_once(granikv_lib, group, schedule, d):
    """bf16, head_dim 128 and 64: each request's suffix items tile its COLD tokens in order, every item is in one run,
    a run's tokens fit the kernel's staging (4096), and every group's pieces are there once."""
    for prefixes, lens, n_q, n_kv in PLANS[group:group + 10]:
        B = len(lens)
        ctx = gb.Context(n_layers=1, n_q=n_q, n_kv=n_kv, head_dim=d, dtype=gb.DTYPE_BF16, n_slots=4_000_000, hot_fraction=0.5,
                         max_batch=B, host_only=True, kv4=True)
        ctx.set_concurrency(*schedule)
        slabs = [ctx.hot_alloc(L)[0] for L in prefixes]
        plan = ctx.dispatch(gb.Batch([slabs[b % len(slabs)] for b in range(B)], lens, 4096, max(lens) + 1))
        img, groups, sched, runs = plan.image(), plan.groups(), plan.schedule(), plan.suffix_runs()
        up = lambda x: (x + 15) // 16 * 16
        at = up(64 * len(groups))
        at = up(at + 4 * B)
        reqs = np.frombuffer(img, np.int32, 4 * B, at).reshape(B, 4)
        at = up(at + 16 * B)
        n_items = sched["prefix_ctas"]
        items = np.frombuffer(img, np.int32, 4 * n_items, at).reshape(n_items, 4)
        assert len({tuple(x) for x in items}) == n_items
        at = up(at + 16 * n_items)
        n_seg = int((reqs[:, 2] - reqs[:, 1]).sum())
        seg = np.frombuffer(img, np.int32, 4 * n_seg, at).reshape(n_seg, 4)
        spans = {}
        for b, t0, t1, _ in seg:
            spans.setdefault(int(b), []).append((int(t0), int(t1)))
        for b, n in enumerate(lens):
            edges = spans.get(b, [])
            assert [e[0] for e in edges] == [0][:len(edges)] + [e[1] for e in edges[:-1]]
            assert (edges[-1][1] if edges else 0) == n and all(t1 > t0 for t0, t1 in edges)
        assert n_items == sum(g["n_splits"] * n_kv * -(-g["m_eff"] // 128) for g in groups)
        begin = np.frombuffer(img, np.int32, runs["runs"] + 1, up(at + 16 * n_seg))
        assert begin[0] == 0 and begin[-1] == n_seg and (np.diff(begin) >= 0).all()
        tokens = np.concatenate([[0], np.cumsum(seg[:, 2] - seg[:, 1])])
        assert (tokens[begin[1:]] - tokens[begin[:-1]]).max(initial=0) <= 4096
        assert runs["tail_runs"] <= n_items and runs["tail_runs"] <= runs["runs"]
