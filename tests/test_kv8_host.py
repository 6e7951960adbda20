"""CPU checks of the 8-bit cache and of eviction: the oracle's number format and selection pinned
by other means, and the refusals of the entry points (checked before any device call)."""

import itertools

import numpy as np
import pytest

import oracle.kv8 as K8
from shared_prefix_kv_decode_gb300 import _binding as gb


def _ctx(kv8=True, n_q=8, n_kv=2, d=64, dtype=gb.DTYPE_BF16, max_batch=8):
    return gb.Context(n_layers=1, n_q=n_q, n_kv=n_kv, head_dim=d, dtype=dtype, n_slots=1000, hot_fraction=0.5,
                      max_batch=max_batch, host_only=True, kv8=kv8)


def _status(call, *args):
    with pytest.raises(gb.GranikvError) as e:
        call(*args)
    return e.value.status


def test_e4m3_codes_match_torch():
    torch = pytest.importorskip("torch")
    codes = torch.arange(256, dtype=torch.uint8)
    assert np.array_equal(codes.view(torch.float8_e4m3fn).float().numpy(), K8.e4m3_values().astype(np.float32), equal_nan=True)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(4096) * 2.0 ** rng.integers(-12, 9, 4096), K8.e4m3_values()[:127],
                        (K8.e4m3_values()[:126] + K8.e4m3_values()[1:127]) / 2]).astype(np.float32)
    x = np.concatenate([x, -x])
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(K8.e4m3_codes(x), want)


def test_quantise_edges():
    x = np.zeros((3, 2, 4), dtype=np.float32)
    x[0, 0] = [1.0, -2.0, np.inf, np.nan]
    x[1, 1] = [3e38, -1e-38, 0.0, 5.0]
    x[2, 0] = 1e-40
    codes, scales = K8.quantise(x, 1)
    assert scales[0, 0] == np.float32(2.0) / np.float32(448) and scales[0, 1] == np.float32(2.0 ** -96) / np.float32(448)
    assert list(codes[0, 0]) == [0x76, 0xFE, 0x7E, 0x7F]  # 224, -448, saturated, NaN
    assert not codes[2, 0].any()  # far below the smallest scale's step
    assert codes[1, 1, 0] == 0x7E and np.isfinite(K8.values(codes[1:2], scales[1:2])).all()
    one, _ = K8.quantise(np.repeat(x[:1, 1:], 65, axis=0), K8.BLOCK)
    assert not one.any()
    y = np.ones((130, 1, 4), dtype=np.float32)
    y[70] = 7.0
    assert [float(s) for s in K8.quantise(y, 64)[1][[0, 63, 64, 127, 128], 0]] == [
        float(np.float32(v) / np.float32(448)) for v in (1, 1, 7, 7, 1)]


def test_evict_oracle_removes_a_lightest_set():
    rng = np.random.default_rng(1)
    for n, e, first, last in [(7, 3, 1, 1), (6, 6, 0, 0), (5, 0, 2, 2), (8, 2, 3, 2)]:
        w = rng.integers(0, 4, (1, 10)).astype(np.float32)
        t = rng.permutation(10)[None].astype(np.int32)
        table, weight, lens, gone = K8.evict([n], [e], [first], last, t, w)
        places = range(first, n - last)
        best = min((sum(w[0, list(c)]) for c in itertools.combinations(places, e)), default=0.0)
        where = [list(t[0]).index(s) for s in gone]
        assert lens == [n - e] and sum(w[0, where]) == best and set(where) <= set(places)
        assert list(table[0, :n - e]) == [s for s in t[0, :n] if s not in set(gone)]
        assert not weight[0, n - e:n].any() and np.array_equal(weight[0, n:], w[0, n:])


@pytest.mark.parametrize("n_kv,d,want", [(8, 128, 1056), (1, 32, 48), (3, 96, 304), (2, 64, 144), (5, 256, 1312)])
def test_row_bytes(granikv_lib, n_kv, d, want):
    assert gb.kv8_row_bytes(n_kv, d) == want


def test_row_bytes_refusals(granikv_lib):
    assert _status(gb.kv8_row_bytes, 0, 64) == gb.ERR_INVALID
    for d in (0, 31, 48, 288):
        assert _status(gb.kv8_row_bytes, 2, d) == gb.ERR_UNSUPPORTED


def test_rows_too_long_are_refused(granikv_lib):
    assert gb.kv8_row_bytes(2 ** 24 // 260, 256) <= 2 ** 24
    for n_kv in (2 ** 24 // 260 + 1, 2 ** 30):
        assert _status(gb.kv8_row_bytes, n_kv, 256) == gb.ERR_UNSUPPORTED
        with pytest.raises(gb.GranikvError) as e:
            _ctx(n_q=n_kv, n_kv=n_kv, d=256)
        assert e.value.status == gb.ERR_UNSUPPORTED


def test_kv8_context_refusals(granikv_lib):
    with pytest.raises(gb.GranikvError) as e:
        _ctx(d=80)
    assert e.value.status == gb.ERR_UNSUPPORTED
    ctx = _ctx()
    sid, _ = ctx.hot_alloc(100)
    assert _status(ctx.hot_fill, 0, sid, 4096, 4096 + 8) == gb.ERR_INVALID  # not on a 16-byte boundary
    assert _status(ctx.hot_fill, 0, sid, 4096, 4096) == gb.ERR_NO_DEVICE
    assert _status(ctx.cold_append, 0, 4098, 4096, 4096, 3) == gb.ERR_INVALID
    assert _status(ctx.cold_append, 0, 4096, 4096, 4096, 3) == gb.ERR_NO_DEVICE
    b = gb.Batch([sid], [3], 4096, 16)
    assert _status(ctx.decode_attention, 0, 4100, b, None, 4096, 4096, 4096, 1 << 20) == gb.ERR_INVALID
    assert _status(ctx.decode_attention, 0, 4096, b, None, 4104, 4096, 4096, 1 << 20) == gb.ERR_INVALID
    assert _status(ctx.decode_attention, 0, 4096, b, None, 4096, 4096, 4096, 1 << 20) == gb.ERR_NO_DEVICE


def test_kv8_dispatch_plans(granikv_lib):
    """The dispatcher works on an 8-bit context: groups by slab, records for every piece and segment."""
    for d in (64, 128):
        ctx = _ctx(d=d)
        sid, _ = ctx.hot_alloc(300)
        plan = ctx.dispatch(gb.Batch([sid, -1, sid], [5, 40, 0], 4096, 64))
        (grp,) = plan.groups()
        assert grp["slab_id"] == sid and grp["n_requests"] == 2 and grp["L_p"] == 300
        assert ctx.workspace_size(plan) > 0


def _plan_case(rng):
    n_prefix = int(rng.choice([1, 1, 2, 5, 20]))
    B = int(rng.choice([1, 2, 7, 40, 200, 1000]))
    prefixes = [int(np.exp(rng.uniform(0, 11))) for _ in range(n_prefix)]
    top = np.exp(rng.uniform(0, 9))
    lens = [int(rng.uniform(0, 40000)) if rng.random() < 0.1 else int(rng.uniform(0, top)) for _ in range(B)]
    n_q, n_kv = [(8, 8), (32, 8), (40, 8), (64, 8), (16, 4), (8, 1), (6, 2), (24, 12), (32, 16)][int(rng.integers(9))]
    return prefixes, lens, n_q, n_kv


PLANS = [_plan_case(np.random.default_rng(s)) for s in range(120)] + [
    ([16384], [300] * 8, 32, 8), ([8192], [250], 32, 8), ([16384], [1] * 64, 32, 8), ([100000], [300000, 1], 32, 8),
    ([100], [200000, 3, 5, 7], 32, 8), ([16384], [100] * 4000, 32, 8), ([500], [0, 1, 2, 3] * 1000, 32, 8)]


@pytest.mark.parametrize("group", range(0, len(PLANS), 10))
@pytest.mark.parametrize("schedule", [(True, 0.0), (True, 0.5), (False, 0.0)])
def test_plans_cover_every_token_once(granikv_lib, group, schedule):
    """Head_dim 128: each request's suffix items tile its COLD tokens in order, every item is in one run,
    a run's tokens fit the kernel's staging (4096), and every group's pieces are there once."""
    for prefixes, lens, n_q, n_kv in PLANS[group:group + 10]:
        B = len(lens)
        ctx = gb.Context(n_layers=1, n_q=n_q, n_kv=n_kv, head_dim=128, dtype=gb.DTYPE_BF16, n_slots=4_000_000, hot_fraction=0.5,
                         max_batch=B, host_only=True, kv8=True)
        ctx.set_concurrency(*schedule)
        slabs = [ctx.hot_alloc(L)[0] for L in prefixes]
        plan = ctx.dispatch(gb.Batch([slabs[b % len(slabs)] for b in range(B)], lens, 4096, max(lens) + 1))
        img, groups, sched, runs = plan.image(), plan.groups(), plan.schedule(), plan.suffix_runs()
        up = lambda x: (x + 15) // 16 * 16
        at = up(64 * len(groups))
        at = up(at + 4 * B)
        reqs = np.frombuffer(img, np.int32, 4 * B, at).reshape(B, 4)
        at = up(at + 16 * B)
        n_items = sum(g["n_splits"] * n_kv * -(-g["m_eff"] // 128) for g in groups)
        assert sched["prefix_ctas"] == n_items
        items = np.frombuffer(img, np.int32, 4 * n_items, at).reshape(n_items, 4)
        assert len({tuple(x) for x in items}) == n_items
        at = up(at + 16 * n_items)
        n_seg = int((reqs[:, 2] - reqs[:, 1]).sum())
        seg = np.frombuffer(img, np.int32, 4 * n_seg, at).reshape(n_seg, 4)
        begin = np.frombuffer(img, np.int32, runs["runs"] + 1, up(at + 16 * n_seg))
        assert begin[0] == 0 and begin[-1] == n_seg and (np.diff(begin) >= 0).all()
        spans = {}
        for b, t0, t1, _ in seg:
            spans.setdefault(int(b), []).append((int(t0), int(t1)))
        for b, n in enumerate(lens):
            edges = spans.get(b, [])
            assert [e[0] for e in edges] == [0][:len(edges)] + [e[1] for e in edges[:-1]]
            assert (edges[-1][1] if edges else 0) == n and all(t1 > t0 for t0, t1 in edges)
        tokens = np.concatenate([[0], np.cumsum(seg[:, 2] - seg[:, 1])])
        assert (tokens[begin[1:]] - tokens[begin[:-1]]).max(initial=0) <= 4096
        assert runs["tail_runs"] <= n_items and runs["tail_runs"] <= runs["runs"]


@pytest.mark.parametrize("kv8", [False, True])
def test_weigh_refusals(granikv_lib, kv8):
    ctx = _ctx(kv8=kv8)
    ok = gb.Batch([-1, -1], [3, 0], 4096, 16, 4096)
    assert _status(ctx.cold_weigh, 0, 4096, 4096, ok, 4096) == gb.ERR_NO_DEVICE
    bad = [
        (1, 4096, 4096, ok, 4096, 1.0),                                         # no such layer
        (0, None, 4096, ok, 4096, 1.0), (0, 4096, None, ok, 4096, 1.0), (0, 4096, 4096, ok, None, 1.0),
        (0, 4100, 4096, ok, 4096, 1.0),                                         # q off its boundary
        (0, 4096, 4096, ok, 4096, -0.5), (0, 4096, 4096, ok, 4096, float("nan")), (0, 4096, 4096, ok, 4096, float("inf")),
        (0, 4096, 4096, gb.Batch([-1], [3], 4096, 16), 4096, 1.0),              # no device lengths
        (0, 4096, 4096, gb.Batch([-1], [17], 4096, 16, 4096), 4096, 1.0),       # past cap
        (0, 4096, 4096, gb.Batch([-1], [-1], 4096, 16, 4096), 4096, 1.0),
        (0, 4096, 4096, gb.Batch([-1] * 9, [1] * 9, 4096, 16, 4096), 4096, 1.0),  # over max_batch
        (0, 4096, 4096, gb.Batch([], [], 4096, 16, 4096), 4096, 1.0),
        (0, 4096, 4096, gb.Batch([-1], [3], None, 16, 4096), 4096, 1.0),
    ]
    for args in bad:
        assert _status(ctx.cold_weigh, *args) == gb.ERR_INVALID, args


def test_evict_refusals(granikv_lib):
    ctx = _ctx()

    def st(lens, out, first, last, table=4096, length=4096, weight=4096, cap=16, slots=4096):
        return _status(ctx.cold_evict, lens, out, first, last, table, length, weight, cap, slots)

    assert st([10], [4], [2], 4) == gb.ERR_NO_DEVICE
    assert st([10], [4], None, 6) == gb.ERR_NO_DEVICE
    for args in [([10], [5], [2], 4), ([10], [-1], [0], 0), ([17], [1], [0], 0), ([-1], [0], [0], 0), ([10], [1], [-1], 0),
                 ([10], [1], [0], -1), ([10], [1], [2 ** 31 - 1], 2 ** 31 - 1), ([4], [1], [9], 0), ([1] * 9, [0] * 9, None, 0),
                 ([], [], None, 0)]:
        assert st(*args) == gb.ERR_INVALID, args
    assert st([10], [1], None, 0, table=None) == gb.ERR_INVALID
    assert st([10], [1], None, 0, weight=None) == gb.ERR_INVALID
    assert st([10], [1], None, 0, slots=None) == gb.ERR_INVALID
    assert st([10], [0], None, 0, slots=None) == gb.ERR_NO_DEVICE
    with pytest.raises(ValueError):
        ctx.cold_evict([1, 2], [0], None, 0, 4096, 4096, 4096, 16, 4096)


def test_host_arrays_are_taken_as_they_are(granikv_lib):
    a = gb.int32_array([3, 1, 2])
    assert gb.int32_array(a) is a and list(a) == [3, 1, 2]


def test_batch_keeps_its_own_counts(granikv_lib):
    """A batch made from a host array does not follow what the caller writes to the array later."""
    slabs, lens = gb.int32_array([-1, -1]), gb.int32_array([3, 2])
    b = gb.Batch(slabs, lens, 4096, 16, 4096)
    live = b.with_live(8192)
    slabs[0], lens[0], lens[1] = 5, 17, -4
    for x in (b, live):
        assert [x.c.slab_id[i] for i in range(2)] == [-1, -1] and [x.c.seq_len[i] for i in range(2)] == [3, 2]
    assert _status(_ctx().cold_weigh, 0, 4096, 4096, b, 4096) == gb.ERR_NO_DEVICE
