"""Decode attention and weighing over the packed caches where scales lie far apart, and calls that follow one another:
against 64 bits on the values held, without the allowance for weights that vanish beside others.

Tolerance of o, with A = sum_t p_t |v_t| of each column over a request's L keys and x the error of a score: a weight is rounded
by half a step of fp16 (2^-11; none in fp32 contexts), products and sums are fp32 (L 2^-24), a score's error moves its weight
by x relative and the sum by as much, the exponential and the merge add 2^-20, all relative to A; then the
rounding to the type (2^-8 or 2^-24).  x = d 2^-24 sum |q_i k_i| / sqrt(d), and what the 8-bit prefix's two parts of q
leave out: 2^-17 of the row's largest q for elements below 2^-9 of it."""

import math

import numpy as np
import pytest

from tests.test_gpu_kv4 import Kv4
from tests.test_gpu_kv8 import Kv8, _gb, _rows, _torch

pytestmark = pytest.mark.gpu

CACHES = {8: Kv8, 4: Kv4}


def _exact(c, b):
    """o [n_kv, g, d] and lse [n_kv, g] of request b in 64 bits, sum p |v|, and a score's error."""
    K, V = c.keys(b)[:2]
    q = c.q_host[b].reshape(c.n_kv, -1, c.d)
    s = np.einsum("jgd,ljd->jgl", q, K) / math.sqrt(c.d)
    x = c.d * 2.0 ** -24 * np.einsum("jgd,ljd->jgl", np.abs(q), np.abs(K)).max(axis=2) / math.sqrt(c.d)
    if isinstance(c, Kv8) and c.of[b] >= 0:
        top = np.abs(q).max(axis=2, keepdims=True)
        small = np.where(np.abs(q) < 2.0 ** -9 * top, np.minimum(np.abs(q), 2.0 ** -17 * top), 0.0)
        x = x + np.einsum("jgd,ljd->jgl", small, np.abs(K)).max(axis=2) / math.sqrt(c.d)
    m = s.max(axis=2, keepdims=True)
    p = np.exp(s - m)
    lse = m[..., 0] + np.log(p.sum(axis=2))
    p /= p.sum(axis=2, keepdims=True)
    return np.einsum("jgl,ljd->jgd", p, V), lse, np.einsum("jgl,ljd->jgd", p, np.abs(V)), x, K.shape[0]


def _check(c, o, lse, what):
    bf16 = c.dtype == "bf16"
    for b in range(len(c.lens)):
        want, want_lse, A, x, L = _exact(c, b)
        tol = (L * 2.0 ** -24 + 2 * x[..., None] + 2.0 ** -20 + (2.0 ** -11 if bf16 else 0.0)) * A
        tol += (2.0 ** -8 if bf16 else 2.0 ** -24) * (np.abs(want) + tol)
        got = o[b].double().cpu().numpy().reshape(want.shape)
        err = np.abs(got - want)
        assert (err <= tol).all(), f"{what} request {b}: o off by {np.nanmax(err / tol)} of its tolerance, NaN {np.isnan(got).any()}"
        err = np.abs(lse[b].double().cpu().numpy().reshape(want_lse.shape) - want_lse)
        tol = x + L * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * np.abs(want_lse)
        assert (err <= tol).all(), f"{what} request {b}: lse off by {np.nanmax(err / tol)} of its tolerance"


SHAPES = [(8, 32, 8, 128, "bf16"), (4, 32, 8, 128, "bf16"), (4, 32, 8, 64, "bf16"), (4, 8, 2, 64, "f32"), (8, 9, 3, 96, "bf16")]


# ---- values far apart ---------------------------------------------------------------------------

@pytest.mark.parametrize("bits,n_q,n_kv,d,dtype", SHAPES)
@pytest.mark.parametrize("e", [6, 9, 16, 24, 33, 45, 100])
@pytest.mark.parametrize("at", [0, 2, 4])
def test_values_beside_a_block_with_a_weightless_outlier(cuda_ok, bits, n_q, n_kv, d, dtype, e, at):
    """One token of a slab block has V of 2^e and no weight (its score is 150 below the others', a weight of 2^-216), the block's
    others have V 0: the output is made of the other blocks' V alone, however far their scales lie below."""
    row = 64 * at + 17

    def edit(kind, k, v):
        k[:, :, 0] = 0.0
        if kind == "prefix":
            v[64 * at:64 * at + 64] = 0.0
            k[row], v[row] = 0.0, np.float32(2.0 ** e)
            k[row, :, 0] = -54.0

    c = CACHES[bits](np.random.default_rng([bits, d, e]), n_q=n_q, n_kv=n_kv, d=d, dtype=dtype, prefixes=[340], of=[0, 0, -1, 0],
                     lens=[0, 30, 5, 1], edit=edit)
    c.q[:, :, 0] = 32.0
    c.q_host[:, :, 0] = 32.0
    _check(c, *c.decode(), f"{bits} bits, 2^{e} in block {at}")


@pytest.mark.parametrize("bits,n_q,n_kv,d,dtype", SHAPES)
@pytest.mark.parametrize("low", [-100, -40, 0, 20])
@pytest.mark.parametrize("span", [7, 9, 30, 80, 106])
def test_values_of_blocks_far_apart(cuda_ok, bits, n_q, n_kv, d, dtype, low, span):
    """Blocks of V about 2^low and 2^(low + span) in turn, the large ones with V in the lower half of the dims and zeros in the
    upper half only: in the upper half the small blocks' V is the whole output.  Many blocks, so that pieces have several.
    (Sums of 2,000 unnormalised weights times V stay within fp32.)"""
    if low + span > 106:
        pytest.skip("V itself would pass fp32")
    def edit(kind, k, v):
        if kind == "prefix":
            at = np.arange(len(v)) // 64 % 2 == 0
            v *= np.float32(2.0 ** low)
            v[at] *= np.float32(2.0 ** span)
            v[at, :, d // 2:] = 0.0
        else:
            v *= np.float32(2.0 ** low)

    c = CACHES[bits](np.random.default_rng([bits, d, span]), n_q=n_q, n_kv=n_kv, d=d, dtype=dtype, prefixes=[2000], of=[0, 0, 0],
                     lens=[0, 3, 40], edit=edit)
    _check(c, *c.decode(), f"{bits} bits, 2^{low} and 2^{span} above")


@pytest.mark.parametrize("bits,d", [(8, 128), (4, 128), (4, 64)])
@pytest.mark.parametrize("zero", ["first", "last", "most"])
def test_values_beside_zero_blocks_in_long_pieces(cuda_ok, bits, d, zero):
    """Pieces of many tiles (160 requests of 64 heads make 80 row blocks) where some blocks' V is all zero."""
    L = 5000

    def edit(kind, k, v):
        if zero == "most":
            v[: 40 * 64], v[42 * 64:] = 0.0, 0.0
        else:
            v[slice(0, 64) if zero == "first" else slice(L // 64 * 64, L)] = 0.0

    c = CACHES[bits](np.random.default_rng([bits, d]), n_q=64, n_kv=8, d=d, dtype="bf16", prefixes=[L], of=[0] * 160, lens=[0] * 160, edit=edit)
    assert c.ctx.dispatch(c.batch).groups()[0]["n_splits"] <= 2
    o, lse = c.decode()
    rows = [0, 1, 15, 16, 17, 80, 158, 159]
    c.of, c.lens, c.q_host = [0] * len(rows), [0] * len(rows), c.q_host[rows]
    c.ck, c.cv = c.ck[:len(rows)], c.cv[:len(rows)]
    if bits == 4:
        c.cu = c.cu[:len(rows)]
    _check(c, o[rows], lse[rows], f"{bits} bits, zeros {zero}")


def _far_apart(kind, k, v):
    if kind == "prefix":
        v[64:128] *= np.float32(2.0 ** 40)
        v[192:] *= np.float32(2.0 ** -40)


@pytest.mark.parametrize("bits,d", [(8, 128), (4, 128), (4, 64)])
@pytest.mark.parametrize("block", [0, 1, 3])
def test_nan_beside_blocks_far_apart(cuda_ok, bits, d, block):
    """A NaN in V stays with its columns (4 bits: the 16 of its scale), one in K or q with the heads that meet it."""
    torch = _torch()
    t = 64 * block + 9

    def case(edit):
        return CACHES[bits](np.random.default_rng([bits, d, 9]), n_q=16, n_kv=4, d=d, dtype="bf16", prefixes=[300], of=[0, 0, -1], lens=[0, 20, 7],
                            edit=lambda kind, k, v: (_far_apart(kind, k, v), edit(kind, k, v)))

    plain = case(lambda kind, k, v: None)
    o, lse = plain.decode()
    _check(plain, o, lse, "without")

    def bad(name):
        def edit(kind, k, v):
            if kind == "prefix":
                (k if name == "k" else v)[t, 1, 37] = np.nan
        return edit

    o2, lse2 = case(bad("v")).decode()
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[:2, 4:8, slice(32, 48) if bits == 4 else 37] = True
    assert torch.equal(torch.isnan(o2), hit) and not torch.isnan(lse2).any()
    o2, lse2 = case(bad("k")).decode()
    hit = torch.zeros_like(lse, dtype=torch.bool)
    hit[:2, 4:8] = True
    assert torch.equal(torch.isnan(lse2), hit) and torch.equal(torch.isnan(o2), hit[..., None].expand_as(o2))
    assert torch.equal(o2[~hit], o[~hit]) and torch.equal(lse2[~hit], lse[~hit])
    for x in (float("nan"), float("inf"), -float("inf")):
        c = case(lambda kind, k, v: None)
        c.q[1, 6, 5] = x
        o2, lse2 = c.decode()
        hit = torch.zeros_like(lse, dtype=torch.bool)
        hit[1, 6] = True
        assert torch.equal(torch.isnan(lse2), hit) and torch.equal(torch.isnan(o2), hit[..., None].expand_as(o2))
        assert torch.equal(o2[~hit], o[~hit]) and torch.equal(lse2[~hit], lse[~hit])


# ---- factors of scores beyond fp32 --------------------------------------------------------------

@pytest.mark.parametrize("bits,n_q,n_kv,d,dtype", [(8, 32, 8, 128, "bf16"), (4, 32, 8, 128, "bf16"), (4, 32, 8, 64, "bf16"),
                                                   (8, 24, 2, 128, "bf16"), (4, 24, 2, 128, "bf16"), (4, 8, 2, 64, "f32")])
@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 60, 2.0 ** 110])
def test_large_queries_over_large_keys_of_other_dims(cuda_ok, bits, n_q, n_kv, d, dtype, size):
    """q and K are large, each in dims where the other is zero: all scores are exactly 0, all weights equal, although the
    product of q's and K's scales may pass fp32."""
    def edit(kind, k, v):
        k *= np.float32(size)
        k[:, :, :16] = 0.0

    c = CACHES[bits](np.random.default_rng([bits, d, 5]), n_q=n_q, n_kv=n_kv, d=d, dtype=dtype, prefixes=[150], of=[0, 0, -1, -1],
                     lens=[0, 20, 33, 1], edit=edit)
    c.q[:, :, 16:] = 0.0
    c.q *= size
    c.q_host = c.q.double().cpu().numpy()
    o, lse = c.decode()
    batch = _gb().Batch([c.slabs[i] if i >= 0 else -1 for i in c.of], c.lens, c.table, c.cap, c.live)
    weight = _torch().zeros(4, c.cap, device="cuda")
    c.ctx.cold_weigh(0, c.q, lse, batch, weight, 0.0)
    c.ctx.sync_status()
    c.q_host = np.zeros_like(c.q_host)  # (the same scores, with no error)
    _check(c, o, lse, f"{bits} bits, {size}")
    for b, n in enumerate(c.lens):
        keys = n + (150 if c.of[b] >= 0 else 0)
        # exp(-lse) over n_q heads: lse to its tolerance above, the exponential and the sum 2^-20 and n_q 2^-24
        tol = n_q / keys * (keys * 2.0 ** -24 + 2.0 ** -19 + 2.0 ** -23 * math.log(keys) + n_q * 2.0 ** -24)
        assert (weight[b, :n].double() - n_q / keys).abs().max().item() <= tol if n else True


# ---- lse of few keys ----------------------------------------------------------------------------

@pytest.mark.parametrize("bits,d,where", [(8, 128, "cold"), (4, 128, "cold"), (4, 64, "cold"), (4, 128, "prefix"), (4, 64, "prefix")])
def test_lse_of_one_key_whose_score_is_one_product(cuda_ok, bits, d, where):
    """One key, and one dim where q and K are not zero: the score takes no addition, and lse is the score.  V is about 1 (its
    largest 2 to 16).  Bounds of the errors, in base 2.  COLD: the row sum is e^2 with an argument below 2 of e, rounded by 2^-24,
    twice: 2^-23; the exponential by 2^-22 of e, 1.45 * 2^-21 in the logarithm; that of a sum in [2^-4, 2^4] by 2^-22.  Prefix:
    three sums below 8 by 2^-22 each, the exponential 1.45 * 2^-22, the logarithm near 7 by 2^-21.  Both: factors of the
    score and the way to base e, 5 * 2^-24 of lse.  None has a preferred sign: over 1,920 heads their root mean square
    is that of errors spread evenly up to the bounds, 3^-1/2 of them."""
    def edit(kind, k, v):
        x = k[:, :, 5].copy()
        k[:] = 0.0
        k[:, :, 5] = x

    B = 60
    c = CACHES[bits](np.random.default_rng([bits, d, 6]), n_q=32, n_kv=8, d=d, dtype="bf16", prefixes=[1], of=[0 if where == "prefix" else -1] * B,
                     lens=[0 if where == "prefix" else 1] * B, edit=edit)
    _, lse = c.decode()
    want = np.stack([_exact(c, b)[1].reshape(-1) for b in range(B)])
    err = np.abs(lse.double().cpu().numpy() - want)
    bounds = [2.0 ** -23, 1.45 * 2.0 ** -21, 2.0 ** -22] if where == "cold" else [2.0 ** -22] * 3 + [1.45 * 2.0 ** -22, 2.0 ** -21]
    bounds = math.log(2) * np.array(bounds)
    assert (err <= bounds.sum() + 5 * 2.0 ** -24 * np.abs(want)).all()
    rms = np.sqrt((bounds ** 2).sum() + (5 * 2.0 ** -24 * want) ** 2)
    assert math.sqrt((err ** 2).mean()) <= math.sqrt((rms ** 2).mean() / 3), math.sqrt((err ** 2).mean())


# ---- reading back -------------------------------------------------------------------------------

@pytest.mark.parametrize("n_kv,d", [(8, 128), (2, 64)])
def test_8_bit_rows_read_back_as_the_nearest_values(cuda_ok, n_kv, d):
    """bf16, bit for bit: code times scale rounded once, over every significand that a bf16 block's largest element may have."""
    torch, gb, rng = _torch(), _gb(), np.random.default_rng([n_kv, d, 8])
    import oracle.kv8 as K8
    N = 400
    rows = torch.from_numpy(_rows(rng, N, n_kv, d, "bf16"))
    top = (1.0 + (torch.arange(N * n_kv) % 128) / 128.0).view(N, n_kv) * 2.0 ** torch.from_numpy(rng.integers(-20, 20, (N, n_kv))).float()
    rows = rows / rows.abs().amax(dim=2, keepdim=True) * top[..., None] * 0.99
    rows[:, :, 3] = top
    x = rows.to(torch.bfloat16).cuda()
    pools = [torch.full((2 * N + 10, gb.kv8_row_bytes(n_kv, d)), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    ctx = gb.Context(n_layers=1, n_q=n_kv, n_kv=n_kv, head_dim=d, dtype=gb.DTYPE_BF16, n_slots=2 * N + 10, k_pools=pools[:1], v_pools=pools[1:],
                     hot_fraction=(N + 5.5) / (2 * N + 10), kv8=True)
    sid, _ = ctx.hot_alloc(N)
    ctx.hot_fill(0, sid, x, x)
    slots = torch.arange(N + 6, 2 * N + 6, dtype=torch.int32, device="cuda")
    ctx.cold_append(0, x, x, slots, N)
    for block in (K8.BLOCK, 1):
        k, v = torch.empty_like(x), torch.empty_like(x)
        if block == 1:
            ctx.cold_read(0, slots, N, k, v)
        else:
            ctx.hot_read(0, sid, 0, N, k, v)
        ctx.sync_status()
        m, e = np.frexp(K8.through_cache(x.float().cpu().numpy(), block))
        want = np.ldexp(np.rint(m * 256.0), e - 8)
        assert np.array_equal(k.double().cpu().numpy(), want) and np.array_equal(v.double().cpu().numpy(), want)


# ---- calls that follow one another --------------------------------------------------------------

@pytest.mark.parametrize("bits,n_q,n_kv,d,dtype", [(8, 32, 8, 128, "bf16"), (4, 32, 8, 128, "bf16"), (4, 32, 8, 64, "bf16"), (4, 8, 2, 64, "f32")])
def test_appends_back_to_back_in_a_graph(cuda_ok, bits, n_q, n_kv, d, dtype):
    """A dozen calls that each write other rows into the same newest slots and attend them, one after the other on one
    workspace, with a prefix that fills the SMs, and replayed: every one's result is that of the same call made alone."""
    torch, rng = _torch(), np.random.default_rng([bits, d, 42])
    B = 64
    lens = [int(n) for n in rng.integers(1, 300, B)]
    c = CACHES[bits](rng, n_q=n_q, n_kv=n_kv, d=d, dtype=dtype, prefixes=[9728 if dtype == "bf16" else 1500], of=[0] * B, lens=lens)
    plan = c.ctx.dispatch(c.batch)
    ws = torch.empty(c.ctx.workspace_size(plan), dtype=torch.uint8, device="cuda")
    calls = [[torch.randn(B, n_kv, d, device="cuda").to(c.tdt) * 2.0 ** (i % 5) for _ in range(2)] for i in range(12)]
    alone = [c.decode(plan=plan, k_new=k, v_new=v) for k, v in calls]
    assert not torch.equal(alone[0][0], alone[1][0])
    outs = [(torch.zeros_like(o), torch.zeros_like(lse)) for o, lse in alone]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        for (k, v), (o, lse) in zip(calls, outs):
            c.ctx.decode_attention_append(0, c.q, k, v, c.batch, plan, o, lse, ws, ws.numel(), s)
    for _ in range(15):
        for o, lse in outs:
            o.zero_()
            lse.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            for _ in range(2):
                g.replay()
        s.synchronize()
        for (o, lse), (o1, lse1) in zip(outs, alone):
            assert torch.equal(o, o1) and torch.equal(lse, lse1)
    c.ctx.sync_status()


@pytest.mark.parametrize("bits,d", [(8, 128), (4, 128), (4, 64)])
@pytest.mark.parametrize("L_p,cold", [(100, 0), (4000, 0), (9728, 300)])
def test_stalled_prefix_wait_is_reported_and_the_context_survives(cuda_ok, bits, d, L_p, cold):
    """The first prefix CTA's wait for V runs out (2 s): every role leaves, the CTA goes on to its COLD run, the call is reported, and the
    next ones give what the one before gave.  Pieces of one tile, of many, and a step with COLD runs behind the prefix."""
    import time
    torch, gb, rng = _torch(), _gb(), np.random.default_rng([bits, d, L_p])
    B = 64 if cold else 3
    c = CACHES[bits](rng, n_q=32, n_kv=8, d=d, dtype="bf16", prefixes=[L_p], of=[0] * B, lens=[int(n) for n in rng.integers(cold // 3, cold + 1, B)])
    plan = c.ctx.dispatch(c.batch)
    o, lse = c.decode(plan)
    c.ctx.inject_stall(True, prefix=True)
    t0 = time.perf_counter()
    with pytest.raises(gb.DeviceCheckFailed):
        c.decode(plan)
    waited = time.perf_counter() - t0
    assert 1.5 <= waited <= 30.0, waited
    for _ in range(2):
        o2, lse2 = c.decode(plan)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    c.ctx.inject_stall(True, prefix=True)
    c.ctx.inject_stall(False)
    c.decode(plan)
