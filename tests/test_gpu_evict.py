"""Eviction of COLD tokens on the GPU: the weight each token received, against 64 bits; which tokens
leave, exactly; and both in a decode loop whose freed slots are used again.

Weights: w = sum_h exp(s_h - lse_h) over n_q heads, all terms positive.  A score's error is at most
x = d 2^-24 sum|q_i k_i| scale (fp32 sum of d products) plus the rounding of s - lse, 2^-23 (|s| + |lse|), in
the exponent; the exponential adds 2^-20 and the sum n_q 2^-24, each relative to w; keep * old adds 2^-23 of it."""

import math

import numpy as np
import pytest

import oracle.kv8 as K8
from tests.test_gpu_kv8 import _gb, _rows, _torch

pytestmark = pytest.mark.gpu


class Cold:
    """COLD rows of a context of either kind, at scattered slots of poisoned pools."""

    def __init__(self, rng, *, n_q, n_kv, d, dtype, lens, kv8, cap=None, q_scale=1.0):
        torch, gb = _torch(), _gb()
        self.n_q, self.n_kv, self.d, self.lens = n_q, n_kv, d, lens
        tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
        total, B = sum(lens), len(lens)
        n_slots = total + 12
        if kv8:
            pools = [torch.full((n_slots, gb.kv8_row_bytes(n_kv, d)), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
        else:
            pools = [torch.full((n_slots, n_kv, d), float("nan"), dtype=tdt, device="cuda") for _ in range(2)]
        self.pools = pools
        self.ctx = gb.Context(n_layers=1, n_q=n_q, n_kv=n_kv, head_dim=d, dtype=gb.DTYPE_BF16 if dtype == "bf16" else gb.DTYPE_F32,
                              n_slots=n_slots, k_pools=[pools[0]], v_pools=[pools[1]], hot_fraction=5.5 / n_slots, max_batch=B, kv8=kv8)
        slots = (5 + rng.permutation(n_slots - 5)[:total]).astype(np.int32)
        k = _rows(rng, total, n_kv, d, dtype)
        self.cap = cap or max(lens) + 2
        table = np.full((B, self.cap), -1, dtype=np.int32)
        self.k, at = [], 0
        for b, n in enumerate(lens):
            table[b, :n] = slots[at:at + n]
            self.k.append((K8.through_cache(k[at:at + n], 1) if kv8 else k[at:at + n]).astype(np.float64))
            at += n
        if total:
            kd = torch.from_numpy(k).cuda().to(tdt)
            self.ctx.cold_append(0, kd, kd, torch.from_numpy(slots).cuda(), total)
        self.table = torch.from_numpy(table).cuda()
        self.live = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.batch = gb.Batch([-1] * B, lens, self.table, self.cap, self.live)
        q = torch.from_numpy((rng.standard_normal((B, n_q, d)) * q_scale).astype(np.float32)).to(tdt)
        self.q, self.q_host = q.cuda(), q.double().numpy()
        self.s = [np.einsum("jgd,ljd->jgl", self.q_host[b].reshape(n_kv, -1, d), self.k[b]).reshape(n_q, -1) / math.sqrt(d) for b in range(B)]
        self.x = [d * 2.0 ** -24 * np.einsum("jgd,ljd->jgl", np.abs(self.q_host[b]).reshape(n_kv, -1, d), np.abs(self.k[b])).reshape(n_q, -1)
                  / math.sqrt(d) for b in range(B)]
        # a lse as of a longer sequence (a prefix took some of the weight)
        lse = np.stack([np.log(np.exp(s).sum(axis=1) + rng.uniform(0, 5)) if s.shape[1] else np.zeros(n_q) for s in self.s])
        self.lse = torch.from_numpy(lse.astype(np.float32)).cuda()
        self.lse_host = self.lse.double().cpu().numpy()

    def check(self, got, before, keep, lens=None, what=""):
        got, before = got.double().cpu().numpy(), before.double().cpu().numpy()
        for b, n in enumerate(lens or self.lens):
            e = self.s[b][:, :n] - self.lse_host[b][:, None]
            p = np.where(np.isneginf(self.lse_host[b])[:, None], 0.0, np.exp(e))
            rel = self.x[b][:, :n] + 2.0 ** -23 * (np.abs(self.s[b][:, :n]) + np.abs(np.where(np.isfinite(self.lse_host[b]), self.lse_host[b], 0))[:, None]) + 2.0 ** -20
            old = keep * before[b, :n] if keep else 0.0
            tol = (p * rel).sum(axis=0) + self.n_q * 2.0 ** -24 * p.sum(axis=0) + 2.0 ** -23 * (np.abs(old) + p.sum(axis=0))
            err = np.abs(got[b, :n] - (p.sum(axis=0) + old))
            assert (err <= tol).all(), f"{what} row {b}: off by {np.max(err / tol)} of the tolerance at {int(np.argmax(err / tol))}"
            assert np.array_equal(got[b, n:], before[b, n:], equal_nan=True), f"{what} row {b}: places past the row changed"


WEIGH = [(32, 8, 128, "bf16"), (40, 8, 128, "bf16"), (7, 1, 128, "bf16"), (6, 3, 128, "bf16"), (64, 4, 128, "bf16"), (8, 2, 64, "f32"), (12, 12, 128, "bf16"),
         (9, 3, 96, "bf16"), (4, 2, 256, "f32"), (64, 64, 32, "f32"), (8, 8, 128, "f32")]


@pytest.mark.parametrize("n_q,n_kv,d,dtype", WEIGH)
@pytest.mark.parametrize("kv8", [False, True])
def test_weigh_matches_64_bit(cuda_ok, n_q, n_kv, d, dtype, kv8):
    torch, rng = _torch(), np.random.default_rng([n_q, n_kv, d, kv8])
    c = Cold(rng, n_q=n_q, n_kv=n_kv, d=d, dtype=dtype, lens=[1, 0, 15, 16, 17, 31, 33, 129, 400, 64], kv8=kv8)
    before = torch.rand(10, c.cap, device="cuda")
    for keep in (1.0, 0.0, 0.9):
        w = before.clone()
        if keep == 0.0:
            for b, n in enumerate(c.lens):
                w[b, :n] = float("nan")  # must not be read
        start = w.clone()
        c.ctx.cold_weigh(0, c.q, c.lse, c.batch, w, keep)
        c.ctx.sync_status()
        c.check(w, start, keep, what=f"keep {keep}")
        again = start.clone()
        c.ctx.cold_weigh(0, c.q, c.lse, c.batch, again, keep)
        assert torch.equal(w[~torch.isnan(w)], again[~torch.isnan(again)])


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("lens", [[1], [5000], [1, 4000, 3], [63] * 70])
def test_weigh_lengths(cuda_ok, kv8, lens):
    torch, rng = _torch(), np.random.default_rng([len(lens), sum(lens)])
    c = Cold(rng, n_q=32, n_kv=8, d=128, dtype="bf16", lens=lens, kv8=kv8)
    w = torch.zeros(len(lens), c.cap, device="cuda")
    start = w.clone()
    c.ctx.cold_weigh(0, c.q, c.lse, c.batch, w, 1.0)
    c.ctx.sync_status()
    c.check(w, start, 1.0)


@pytest.mark.parametrize("kv8", [False, True])
def test_weigh_live_lengths_stream_and_graph(cuda_ok, kv8):
    """Captured once, replayed with other device lengths, q and lse on another stream."""
    torch, rng = _torch(), np.random.default_rng(3)
    c = Cold(rng, n_q=32, n_kv=8, d=128, dtype="bf16", lens=[40, 90, 7], kv8=kv8)
    w = torch.rand(3, c.cap, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.ctx.cold_weigh(0, c.q, c.lse, c.batch, w, 1.0, s)
    for live in ([40, 90, 7], [13, 0, 7], [400, 1, 2]):
        c.live.copy_(torch.tensor(live, dtype=torch.int32))
        before = w.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        s.synchronize()
        c.check(w, before, 1.0, [min(a, b) for a, b in zip(live, c.lens)], f"live {live}")
    c.ctx.sync_status()


@pytest.mark.parametrize("kv8", [False, True])
def test_weigh_empty_head_and_bad_slot(cuda_ok, kv8):
    torch, gb, rng = _torch(), _gb(), np.random.default_rng(4)
    c = Cold(rng, n_q=32, n_kv=8, d=128, dtype="bf16", lens=[40, 20], kv8=kv8)
    c.lse[0, 3] = float("-inf")
    c.lse_host[0, 3] = -np.inf
    w = torch.zeros(2, c.cap, device="cuda")
    c.ctx.cold_weigh(0, c.q, c.lse, c.batch, w, 1.0)
    c.ctx.sync_status()
    c.check(w, torch.zeros_like(w), 1.0)
    c.table[1, 5] = c.pools[0].shape[0]
    before = torch.rand(2, c.cap, device="cuda")
    w = before.clone()
    c.ctx.cold_weigh(0, c.q, c.lse, c.batch, w, 0.5)
    with pytest.raises(gb.DeviceCheckFailed):
        c.ctx.sync_status()
    assert w[1, 5] == 0.5 * before[1, 5]
    c.table[1, 5] = c.table[1, 6]
    w[1, 5] = before[1, 5]
    keep = [i for i in range(20) if i != 5]
    ref = before.clone()
    c.ctx.cold_weigh(0, c.q, c.lse, c.batch, ref, 0.5)
    assert torch.equal(ref[1, keep], w[1, keep])


@pytest.mark.parametrize("kv8", [False, True])
def test_weigh_more_rows_than_one_launch(cuda_ok, kv8):
    torch, rng = _torch(), np.random.default_rng(6)
    lens = [int(x) for x in rng.integers(0, 6, 1030)]
    lens[1023], lens[1024], lens[1029] = 70, 65, 3
    c = Cold(rng, n_q=8, n_kv=2, d=128, dtype="bf16", lens=lens, kv8=kv8)
    w = torch.rand(len(lens), c.cap, device="cuda")
    start = w.clone()
    kernels, _ = c.ctx.launch_count()
    c.ctx.cold_weigh(0, c.q, c.lse, c.batch, w, 0.5)
    c.ctx.sync_status()
    assert c.ctx.launch_count()[0] == kernels + 2
    c.check(w, start, 0.5)


def test_weigh_bad_query_stays_with_its_row(cuda_ok):
    """A NaN in one request's q makes its tokens' weights NaN (the last to leave) and changes no other row."""
    torch, rng = _torch(), np.random.default_rng(7)
    for kv8 in (False, True):
        c = Cold(rng, n_q=32, n_kv=8, d=128, dtype="bf16", lens=[100, 40, 70], kv8=kv8)
        w = torch.zeros(3, c.cap, device="cuda")
        c.ctx.cold_weigh(0, c.q, c.lse, c.batch, w, 1.0)
        bad = torch.zeros(3, c.cap, device="cuda")
        c.q[1, 9, 3] = float("nan")
        c.ctx.cold_weigh(0, c.q, c.lse, c.batch, bad, 1.0)
        c.ctx.sync_status()
        assert torch.isnan(bad[1, :40]).all() and not torch.isnan(bad[1, 40:]).any()
        assert torch.equal(bad[[0, 2]], w[[0, 2]])


def test_weights_of_a_step_sum_to_the_heads(cuda_ok):
    """Weighed with decode's own lse and no prefix, a request's tokens share the n_q heads' weight of 1."""
    torch, gb, rng = _torch(), _gb(), np.random.default_rng(5)
    for kv8 in (False, True):
        c = Cold(rng, n_q=32, n_kv=8, d=128, dtype="bf16", lens=[100, 1, 700], kv8=kv8)
        plan = c.ctx.dispatch(c.batch)
        ws = torch.empty(c.ctx.workspace_size(plan), dtype=torch.uint8, device="cuda")
        o, lse = torch.empty_like(c.q), torch.empty(3, 32, device="cuda")
        c.ctx.decode_attention(0, c.q, c.batch, plan, o, lse, ws, ws.numel())
        w = torch.zeros(3, c.cap, device="cuda")
        c.ctx.cold_weigh(0, c.q, lse, c.batch, w, 0.0)
        c.ctx.sync_status()
        assert torch.allclose(w.sum(dim=1), torch.full((3,), 32.0, device="cuda"), rtol=1e-4)


# ---- eviction ---------------------------------------------------------------------------------

def _evict_ctx(B):
    torch, gb = _torch(), _gb()
    pool = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    ctx = gb.Context(n_layers=1, n_q=1, n_kv=1, head_dim=32, dtype=gb.DTYPE_BF16, n_slots=8, k_pools=[pool], v_pools=[pool], max_batch=B)
    ctx.pool = pool
    return ctx


def _evict_case(rng, lens, out, first, last, cap, weights, rows_after=2, suffix=True):
    torch = _torch()
    B = len(lens)
    ctx = _evict_ctx(B)
    table = rng.permutation((B + rows_after) * cap).reshape(B + rows_after, cap).astype(np.int32)
    w = weights((B + rows_after, cap)).astype(np.float32)
    t_dev, w_dev = torch.from_numpy(table).cuda(), torch.from_numpy(w).cuda()
    length = torch.full((B + rows_after,), -7, dtype=torch.int32, device="cuda")
    slots = torch.full((sum(out) + 3,), -9, dtype=torch.int32, device="cuda")
    ctx.cold_evict(lens, out, first, last, t_dev, length if suffix else None, w_dev, cap, slots)
    ctx.sync_status()
    table, w, new, gone = K8.evict(lens, out, first, last, table, w)
    assert np.array_equal(slots.cpu().numpy(), np.concatenate([gone, [-9] * 3]))
    assert np.array_equal(t_dev.cpu().numpy(), table)
    got = w_dev.cpu().numpy()
    assert np.array_equal(got, w, equal_nan=True)
    assert length.cpu().tolist() == (new if suffix else [-7] * B) + [-7] * rows_after


KINDS = {
    "softmax": lambda rng: lambda shape: np.exp(2.5 * rng.standard_normal(shape) - 6),
    "equal": lambda rng: lambda shape: np.full(shape, 0.25),
    "few": lambda rng: lambda shape: rng.integers(0, 3, shape) / 4.0,
    "zeros": lambda rng: lambda shape: np.where(rng.random(shape) < 0.5, 0.0, -0.0),
    "signed": lambda rng: lambda shape: rng.standard_normal(shape) * 10.0 ** rng.integers(-30, 30, shape),
    "odd": lambda rng: lambda shape: rng.choice([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45, 3.4e38, 1.0], shape),
    "neighbours": lambda rng: lambda shape: np.ones(shape, np.float32).view(np.int32).__add__(rng.integers(0, 300, shape).astype(np.int32)).view(np.float32),
}


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_evict_weights(cuda_ok, kind):
    rng = np.random.default_rng(7)
    lens = [1, 2, 31, 32, 33, 100, 1023, 1024, 1025, 2500, 0, 40]
    first = [0, 1, 0, 4, 4, 50, 3, 0, 1, 100, 0, 40]
    out = [min(max(0, n - f - 5), x) for n, f, x in zip(lens, first, [1, 1, 31, 3, 28, 17, 1000, 511, 1, 1700, 0, 9])]
    _evict_case(rng, lens, out, first, 5, 2504, KINDS[kind](rng))


@pytest.mark.parametrize("n", [1, 1000, 1024, 2049, 4096, 5000, 16385, 20000, 70001, 131073])
@pytest.mark.parametrize("share", [0.0, 0.001, 0.5, 1.0])
def test_evict_lengths(cuda_ok, n, share):
    rng = np.random.default_rng(n)
    out = [max(1 if share else 0, int(n * share)), 0, 1]
    _evict_case(rng, [n, n, n], out, None, 0, n + 5, KINDS["softmax"](rng))


@pytest.mark.parametrize("kind", ["equal", "odd", "few"])
@pytest.mark.parametrize("n", [5000, 40000, 100000, 140000])
def test_evict_ties_across_slices(cuda_ok, kind, n):
    """Long rows of few different weights: the ties that leave are the lowest places of the whole row."""
    rng = np.random.default_rng([n, len(kind)])
    _evict_case(rng, [n, n - 77, 3], [n // 3, n - 200, 2], [5, 0, 0], 0, n, KINDS[kind](rng))


def test_evict_many_middling_rows(cuda_ok):
    """Enough rows of a few thousand tokens that a thread holds eight of them."""
    rng = np.random.default_rng(12)
    lens = [int(x) for x in rng.integers(1500, 5000, 200)]
    _evict_case(rng, lens, [n // 4 for n in lens], [4] * 200, 32, 5000, KINDS["softmax"](rng))


def test_evict_many_rows(cuda_ok):
    """More rows than one launch's parameters hold, and no lengths array."""
    rng = np.random.default_rng(8)
    lens = [int(x) for x in rng.integers(0, 60, 2500)]
    out = [int(rng.integers(0, n + 1)) for n in lens]
    _evict_case(rng, lens, out, None, 0, 60, KINDS["few"](rng), suffix=False)


def test_evict_whole_rows_and_nothing(cuda_ok):
    rng = np.random.default_rng(9)
    _evict_case(rng, [50, 50, 7], [50, 0, 7], None, 0, 50, KINDS["softmax"](rng))
    _evict_case(rng, [50, 0], [0, 0], [3, 0], 4, 64, KINDS["softmax"](rng))


def test_evict_in_a_graph(cuda_ok):
    """Captured with host arrays that are gone at replay, replayed on fresh contents."""
    torch, rng = _torch(), np.random.default_rng(10)
    lens, out, cap = [300, 1200, 5], [100, 700, 5], 1300
    ctx = _evict_ctx(3)
    table = rng.permutation(3 * cap).reshape(3, cap).astype(np.int32)
    t0 = torch.from_numpy(table).cuda()
    t, w = t0.clone(), torch.zeros(3, cap, device="cuda")
    length, slots = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(805, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ctx.cold_evict(list(lens), list(out), None, 0, t, length, w, cap, slots, s)
    for i in range(3):
        wh = rng.random((3, cap)).astype(np.float32)
        t.copy_(t0)
        w.copy_(torch.from_numpy(wh))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        s.synchronize()
        rt, rw, rl, rg = K8.evict(lens, out, None, 0, table, wh)
        assert np.array_equal(t.cpu().numpy(), rt) and np.array_equal(w.cpu().numpy(), rw)
        assert length.cpu().tolist() == rl and np.array_equal(slots.cpu().numpy(), rg)


# ---- together ---------------------------------------------------------------------------------

def test_cache_evict_keeps_shared_slots_and_reuses_the_rest(cuda_ok):
    """A prefix placed in COLD is shared by two requests: eviction never takes its slots, and the
    slots that did leave are allocated again."""
    torch, gb = _torch(), _gb()
    from shared_prefix_kv_decode_gb300 import GraniKVCache
    rng = np.random.default_rng(11)
    cache = GraniKVCache(n_layers=1, n_q=32, n_kv=8, head_dim=128, dtype=gb.DTYPE_BF16, n_slots=600, max_batch=2, cap=300, hot_fraction=0.1, kv8=True)
    x = torch.from_numpy(_rows(rng, 200, 8, 128, "bf16")).cuda().to(torch.bfloat16)
    info, _ = cache.admit([5] * 100, [x[:100]], [x[:100]])
    assert info["slab_id"] == -1
    for b in range(2):
        assert cache.attach(b, [5] * 100 + [7]) == (-1, 100)
    cache.append([60, 40], [x[100:]], [x[100:]])
    batch = cache.batch([-1, -1])
    q = torch.randn(2, 32, 128, device="cuda").to(torch.bfloat16)
    o, lse = cache.decode(0, q, batch)
    cache.weigh(0, q, lse, batch)
    free = cache.ctx.cold_free_count()
    before = cache.req_to_slot.clone()
    with pytest.raises(gb.GranikvError):
        cache.evict([61, 0])
    slots = cache.evict([50, 10], keep_last=4)
    cache.ctx.sync_status(cache.stream())
    assert cache.ctx.cold_free_count() == free + 60 and cache.seq_len_host[:2] == [110, 130]
    assert cache.suffix_len.tolist() == [110, 130]
    for b in range(2):
        assert torch.equal(cache.req_to_slot[b, :100], before[b, :100])
        n = 160 - 20 * b
        assert torch.equal(cache.req_to_slot[b, cache.seq_len_host[b] - 4:cache.seq_len_host[b]], before[b, n - 4:n])
    held = set(cache.req_to_slot[0, :110].tolist()) | set(cache.req_to_slot[1, :130].tolist())
    gone = slots.tolist()
    assert len(set(gone)) == 60 and not held & set(gone)
    # everything that is free can be handed out again, the evicted slots among it
    n = cache.ctx.cold_free_count()
    again = torch.cat([cache.alloc([min(n, 300 - 110), 0]), cache.alloc([0, min(max(0, n - 190), 300 - 130)])]).tolist()
    assert len(set(again)) == len(again) and not held & set(again)
    cache.ctx.sync_status(cache.stream())
    assert not cache.weight[0, 110:].any() and not cache.weight[1, 130:].any()
    cache.detach(0)
    assert not cache.weight[0].any()


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("graph", [False, True])
def test_driver_with_a_cold_budget(cuda_ok, kv8, graph):
    """Steps with arrivals, completions and a budget: every request stays within it, the ring
    accounts for every token, and the last step's attention equals 64-bit attention over exactly the
    tokens that stayed."""
    from oracle import attention as OA
    from shared_prefix_kv_decode_gb300.decode_driver import DecodeDriver

    n_q, n_kv, d, n_slots = 32, 8, 128, 40000
    drv = DecodeDriver(prefix_lens=[700, 300], n_layers=2, n_q=n_q, n_kv=n_kv, head_dim=d, max_batch=32, cap=512, n_slots=n_slots, seed=5,
                       keep_logical=True, graph=graph, headroom=4, kv8=kv8, cold_budget=40, keep_last=8)
    sched = np.random.default_rng(9)
    for i in range(10):
        drv.arrive(i % 2, int(sched.integers(1, 120)))
    for step in range(12):
        if step in (4, 9):
            drv.complete(int(sched.integers(drv.B)))
            drv.arrive(int(sched.integers(2)), int(sched.integers(1, 120)))
        drv.step()
        assert all(r["len"] <= 41 for r in drv.rows)
    trace = drv.finish_trace()
    assert sum(t["evicted"] for t in trace) > 100
    if graph:
        assert sum(t["mode"] == "replay" for t in trace) >= 4
    drv._sync_cold()
    held = sum(r["len"] for r in drv.rows)
    assert held == sum(drv.cache.seq_len_host[:drv.B]) == int(drv.cache.suffix_len[:drv.B].sum())
    assert drv.cache.ctx.cold_free_count() == n_slots - drv.cache.n_hot - held
    o, lse = (x.double().cpu().numpy() for x in drv.last_out)
    q = drv.last_q[1]
    for b in range(drv.B):
        r = drv.rows[b]
        pk, pv = (x.copy() for x in drv.prefix_kv[r["prefix"]][0:2])
        pk, pv = pk[1], pv[1]
        k, v = np.concatenate(r["k"][1], axis=0), np.concatenate(r["v"][1], axis=0)
        assert k.shape[0] == r["len"]
        if kv8:
            pk, pv, k, v = K8.through_cache(pk, 64), K8.through_cache(pv, 64), K8.through_cache(k, 1), K8.through_cache(v, 1)
        K, V = np.concatenate([pk, k]).astype(np.float64), np.concatenate([pv, v]).astype(np.float64)
        for h in range(n_q):
            ref, ref_lse = OA.attend(q[b, h].astype(np.float64), K[:, h // 4], V[:, h // 4], OA.softmax_scale(d))
            # weights in bf16 or fp16 (2^-8 of sum p|v| at most) and the output in bf16 (2^-8 of itself)
            A = np.abs(V[:, h // 4]).max()
            assert np.abs(o[b, h] - ref).max() <= 2.0 ** -8 * (A + np.abs(ref).max()) and abs(lse[b, h] - ref_lse) <= 1e-3


def test_weights_are_not_made_inside_a_capture(cuda_ok):
    """Made while a graph is captured, the weights would be zeroed by every replay: refused, and once they are
    made the captured weighing accumulates over the replays."""
    torch, gb = _torch(), _gb()
    from shared_prefix_kv_decode_gb300 import GraniKVCache
    rng = np.random.default_rng(13)
    cache = GraniKVCache(n_layers=1, n_q=8, n_kv=2, head_dim=128, dtype=gb.DTYPE_BF16, n_slots=400, max_batch=2, cap=64)
    x = torch.from_numpy(_rows(rng, 50, 2, 128, "bf16")).cuda().to(torch.bfloat16)
    cache.append([30, 20], [x], [x])
    batch = cache.batch([-1, -1])
    q = torch.randn(2, 8, 128, device="cuda").to(torch.bfloat16)
    o, lse = cache.decode(0, q, batch)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="before the capture"):
        with torch.cuda.graph(g):
            o.add_(0.0)
            cache.weigh(0, q, lse, batch)
    assert not cache.weight.any()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.weigh(0, q, lse, batch)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.allclose(cache.weight.sum(dim=1), torch.full((2,), 24.0, device="cuda"), rtol=1e-4)


@pytest.mark.parametrize("n_q,n_kv", [(8, 2), (32, 8), (24, 2), (7, 1), (64, 64), (65, 65)])
@pytest.mark.parametrize("kv8", [False, True])
def test_weigh_bf16_heads_of_64(cuda_ok, n_q, n_kv, kv8):
    """On tensor cores up to 64 KV heads; one more, on CUDA cores."""
    torch, rng = _torch(), np.random.default_rng([n_q, n_kv, 64, kv8])
    c = Cold(rng, n_q=n_q, n_kv=n_kv, d=64, dtype="bf16", lens=[1, 0, 15, 16, 17, 31, 33, 129, 400, 64], kv8=kv8)
    before = torch.rand(10, c.cap, device="cuda")
    for keep in (1.0, 0.0):
        w = before.clone()
        c.ctx.cold_weigh(0, c.q, c.lse, c.batch, w, keep)
        c.ctx.sync_status()
        c.check(w, before, keep, what=f"keep {keep}")


@pytest.mark.parametrize("B,n", [(400, 2048), (76, 4000), (77, 4000), (38, 8000), (39, 8000), (8, 16000)])
def test_evict_around_one_wave(cuda_ok, B, n):
    """Rows that take one, two, four or eight CTAs at two tokens a thread, on either side of what 152 SMs run at once."""
    rng = np.random.default_rng([B, n])
    _evict_case(rng, [n - b % 5 for b in range(B)], [n // 3 - b for b in range(B)], None, 7, n, KINDS["few" if B % 2 else "softmax"](rng))
