"""The 8-bit cache on the GPU: what the writes put into the pools, bit for bit, and decode attention
over it against 64-bit attention on the dequantised values.

Every pool starts as 0xff bytes (NaN codes, NaN scales), so anything read outside the written slots
poisons the result.

Tolerances.  With A = sum_t p_t |v_t| (64 bits) over a row's L keys:
  o:   the weights are rounded to fp16 at most (half a step: 2^-11 relative), products and sums are
       fp32, whose error over L terms is at most L 2^-24 relative to A, the normalisation and merge
       add a few 2^-24; an error of x in a score moves its weight by x relative (below).  The result
       is rounded to bf16 (2^-8 relative to it) or kept in fp32.  An fp16 weight P = 2^7 p vs / M, with vs the
       token's V scale and M = max_t p_t vs_t (the kernel may carry more than 2^7, never less), that falls
       below 2^-14 is off by at most half of fp16's last subnormal, 2^-25: by 2^-32 M in p vs, which meets
       a code of at most 448.  With B_t = 448 vs_t, the largest |v| of the token's block and head, that is
       2^-32 max_t(p_t B_t) for each of the L tokens (it shows only where a column's result is
       that far below the row's largest possible one).
  lse: a score q.k is a sum of d exact products in fp32: error at most d 2^-24 sum|q_i k_i| scale; the
       tensor-core prefix takes q as two e4m3 parts, exact but for elements below 2^-9 of the row's largest,
       which are off by at most 2^-17 of that: 2^-17 max|q| sum|k_i| scale over those elements more.
       x is the sum of the two;
       the exponential and logarithm add 2^-20, the sum of L weights L 2^-24.
fp32 contexts keep the weights in fp32, and so have no 2^-11."""

import math

import numpy as np
import pytest

import oracle.kv8 as K8

pytestmark = pytest.mark.gpu


def _gb():
    from shared_prefix_kv_decode_gb300 import _binding as gb
    return gb


def _torch():
    import torch
    return torch


def _rows(rng, n, n_kv, d, dtype, spread=0.5):
    """float32 rows exact in dtype, a few channels larger than the rest."""
    torch = _torch()
    x = rng.standard_normal((n, n_kv, d)) * np.exp(spread * rng.standard_normal((n_kv, d)))
    x = torch.from_numpy(x.astype(np.float32))
    return (x.to(torch.bfloat16).float() if dtype == "bf16" else x).numpy()


class Kv8:
    """An 8-bit context with poisoned pools, its prefixes in slabs and its COLD rows at scattered slots."""

    def __init__(self, rng, *, n_q, n_kv, d, dtype, prefixes=(), of=(), lens=(), cap=None, n_layers=1, slots_before=0,
                 spread=0.5, q_scale=None, holes=7, backend=None, dev=0, edit=None):
        torch, gb = _torch(), _gb()
        self.n_q, self.n_kv, self.d, self.dtype = n_q, n_kv, d, dtype
        self.tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.prefixes, self.of, self.lens = list(prefixes), list(of), list(lens)
        B = len(self.lens)
        n_cold = sum(lens) + holes
        n_hot = slots_before + sum(prefixes) + holes
        n_slots = n_hot + n_cold
        self.row = gb.kv8_row_bytes(n_kv, d)
        self.kp, self.vp = (torch.full((n_slots, self.row), 0xFF, dtype=torch.uint8, device=f"cuda:{dev}") for _ in range(2))
        self.ctx = gb.Context(n_layers=1, n_q=n_q, n_kv=n_kv, head_dim=d, dtype=gb.DTYPE_BF16 if dtype == "bf16" else gb.DTYPE_F32,
                              n_slots=n_slots, k_pools=[self.kp], v_pools=[self.vp], hot_fraction=(n_hot + 0.5) / n_slots,
                              max_batch=max(B, 1), device=dev, kv8=True)
        if backend is not None:
            self.ctx.force_backend(backend)
        if slots_before:
            self.ctx.hot_alloc(slots_before)
        self.dev = self.kp.device
        self.slabs, self.pk, self.pv = [], [], []
        for L in self.prefixes:
            k, v = _rows(rng, L, n_kv, d, dtype, spread), _rows(rng, L, n_kv, d, dtype, spread)
            if edit:
                edit("prefix", k, v)
            sid, _ = self.ctx.hot_alloc(L)
            self.ctx.hot_fill(0, sid, self.to(k), self.to(v))
            self.slabs.append(sid)
            self.pk.append(K8.through_cache(k, K8.BLOCK))
            self.pv.append(K8.through_cache(v, K8.BLOCK))
        self.n_hot = n_hot
        slots = n_hot + rng.permutation(n_cold)[: sum(lens)].astype(np.int32)
        self.cap = cap or max([1] + [n + 3 for n in lens])
        table = np.full((B, self.cap), -1, dtype=np.int32)
        self.ck, self.cv, at = [], [], 0
        for b, n in enumerate(self.lens):
            table[b, :n] = slots[at:at + n]
            at += n
            k, v = _rows(rng, n, n_kv, d, dtype, spread), _rows(rng, n, n_kv, d, dtype, spread)
            if edit:
                edit("cold", k, v)
            if n:
                self.ctx.cold_append(0, self.to(k), self.to(v), torch.from_numpy(table[b, :n].copy()).to(self.dev), n)
            self.ck.append(K8.through_cache(k, 1))
            self.cv.append(K8.through_cache(v, 1))
        self.table = torch.from_numpy(table).to(self.dev)
        self.live = torch.tensor(self.lens, dtype=torch.int32, device=self.dev)
        self.batch = gb.Batch([self.slabs[i] if i >= 0 else -1 for i in self.of], self.lens, self.table, self.cap)
        q = torch.from_numpy((rng.standard_normal((B, n_q, d)) * (q_scale or 1.0)).astype(np.float32)).to(self.tdt)
        self.q_host = q.float().numpy().astype(np.float64)
        self.q = q.to(self.dev)

    def to(self, x):
        return _torch().from_numpy(x).to(self.dev).to(self.tdt)

    def decode(self, plan=None, batch=None, stream=None, k_new=None, v_new=None):
        torch = _torch()
        batch = batch or self.batch
        plan = plan or self.ctx.dispatch(batch)
        n = self.ctx.workspace_size(plan)
        self.ws = torch.empty(n, dtype=torch.uint8, device=self.dev)
        o = torch.full_like(self.q, float("nan"))
        lse = torch.full(self.q.shape[:2], float("nan"), device=self.dev)
        if k_new is None:
            self.ctx.decode_attention(0, self.q, batch, plan, o, lse, self.ws, n, stream)
        else:
            self.ctx.decode_attention_append(0, self.q, k_new, v_new, batch, plan, o, lse, self.ws, n, stream)
        self.ctx.sync_status(stream)
        return o, lse

    def keys(self, b):
        k, v = [self.ck[b]], [self.cv[b]]
        if self.of[b] >= 0:
            k.insert(0, self.pk[self.of[b]])
            v.insert(0, self.pv[self.of[b]])
        return np.concatenate(k), np.concatenate(v)

    def check(self, o, lse, what=""):
        o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
        g = self.n_q // self.n_kv
        for b in range(len(self.lens)):
            K, V = self.keys(b)
            L = K.shape[0]
            q = self.q_host[b].reshape(self.n_kv, g, self.d)
            s = np.einsum("jgd,ljd->jgl", q, K) / math.sqrt(self.d)
            x = self.d * 2.0 ** -24 * (np.einsum("jgd,ljd->jgl", np.abs(q), np.abs(K)) / math.sqrt(self.d)).max(axis=2)
            if self.of[b] >= 0 and self.dtype == "bf16" and self.d == 128:
                top_q = np.abs(q).max(axis=2, keepdims=True)
                small = np.where(np.abs(q) < 2.0 ** -9 * top_q, 2.0 ** -17 * top_q, 0.0)
                x = x + (np.einsum("jgd,ljd->jgl", small, np.abs(K)) / math.sqrt(self.d)).max(axis=2)
            m = s.max(axis=2, keepdims=True)
            p = np.exp(s - m)
            ref_lse = (m[..., 0] + np.log(p.sum(axis=2))).reshape(self.n_q)
            p /= p.sum(axis=2, keepdims=True)
            ref = np.einsum("jgl,ljd->jgd", p, V)
            A = np.einsum("jgl,ljd->jgd", p, np.abs(V))
            n_p = self.pk[self.of[b]].shape[0] if self.of[b] >= 0 else 0
            top = np.abs(V).max(axis=2)
            for t in range(0, n_p, K8.BLOCK):
                top[t:min(t + K8.BLOCK, n_p)] = top[t:min(t + K8.BLOCK, n_p)].max(axis=0)
            floor = 2.0 ** -32 * L * (p * top.T[:, None]).max(axis=2)[..., None] if self.dtype == "bf16" else 0.0
            rel = L * 2.0 ** -24 + 2 * x[..., None] + 2.0 ** -20 + (2.0 ** -11 if self.dtype == "bf16" else 0)
            tol = rel * A + floor
            tol += (2.0 ** -8 if self.dtype == "bf16" else 2.0 ** -24) * (np.abs(ref) + tol)
            err = np.abs(o[b].reshape(ref.shape) - ref)
            if not (err <= tol).all():
                raise AssertionError(f"{what} request {b}: o off by {np.max(err / tol)} of its tolerance ({err.max()})")
            ltol = (x + L * 2.0 ** -24 + 2.0 ** -20).reshape(self.n_q) + 2.0 ** -23 * np.abs(ref_lse)
            lerr = np.abs(lse[b] - ref_lse)
            if not (lerr <= ltol).all():
                raise AssertionError(f"{what} request {b}: lse off by {np.max(lerr / ltol)} of its tolerance")


# ---- writes -----------------------------------------------------------------------------------

def _odd_values(rng, x):
    """Zeros, tiny and huge values, infinities and NaN among the rows."""
    n, n_kv, d = x.shape
    x[0, 0] = 0.0
    if n > 2:
        x[1, :, : d // 2] = 1e-37
        x[2, -1, 0], x[2, -1, 1] = np.inf, -np.inf
    if n > 70:
        x[66, 0, 3] = np.nan
        x[69] *= np.float32(2.0 ** 60)
        x[n - 1] *= np.float32(2.0 ** -120)
    return x


SHAPES = [(8, 128, "bf16"), (2, 64, "f32"), (1, 32, "bf16"), (3, 96, "f32"), (5, 160, "bf16"), (2, 256, "f32"), (4, 192, "bf16"), (1, 224, "f32")]


@pytest.mark.parametrize("n_kv,d,dtype", SHAPES)
@pytest.mark.parametrize("L", [1, 63, 64, 65, 200])
def test_slab_write_is_bit_exact(cuda_ok, n_kv, d, dtype, L):
    torch, rng = _torch(), np.random.default_rng([L, n_kv, d])
    c = Kv8(rng, n_q=n_kv, n_kv=n_kv, d=d, dtype=dtype, slots_before=13)
    k, v = (_odd_values(rng, _rows(rng, L, n_kv, d, dtype)) for _ in range(2))
    k, v = (c.to(x).float().cpu().numpy() for x in (k, v))  # exact in dtype
    # the pools of this context have 13 + 7 HOT slots: a wider one
    gb = _gb()
    n_slots = L + 40
    pools = [torch.full((n_slots, c.row), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    ctx = gb.Context(n_layers=1, n_q=n_kv, n_kv=n_kv, head_dim=d, dtype=c.ctx.dtype, n_slots=n_slots, k_pools=[pools[0]],
                     v_pools=[pools[1]], hot_fraction=(L + 20.5) / n_slots, kv8=True)
    ctx.hot_alloc(13)
    sid, off = ctx.hot_alloc(L)
    assert off == 13
    ctx.hot_fill(0, sid, c.to(k), c.to(v))
    ctx.sync_status()
    for pool, x in zip(pools, (k, v)):
        got = pool.cpu().numpy()
        codes, scales = K8.quantise(x, K8.BLOCK)
        live = got[13:13 + L]
        assert np.array_equal(live[:, : n_kv * d].reshape(L, n_kv, d) & 0x7F, codes & 0x7F)
        same = (live[:, : n_kv * d].reshape(L, n_kv, d) == codes) | ((codes & 0x7F) == 0x7F)
        assert same.all()
        assert np.array_equal(live[:, n_kv * d : n_kv * (d + 4)].copy().view(np.float32), scales)
        rest = np.concatenate([got[:13], got[13 + L:]])
        assert (rest == 0xFF).all() and (live[:, n_kv * (d + 4):] == 0xFF).all()


@pytest.mark.parametrize("n_kv,d,dtype", SHAPES)
@pytest.mark.parametrize("N", [1, 3, 75])
def test_token_write_is_bit_exact(cuda_ok, n_kv, d, dtype, N):
    torch, gb, rng = _torch(), _gb(), np.random.default_rng([N, n_kv, d])
    c = Kv8(rng, n_q=n_kv, n_kv=n_kv, d=d, dtype=dtype)
    n_slots = 2 * N + 30
    pools = [torch.full((n_slots, c.row), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    ctx = gb.Context(n_layers=1, n_q=n_kv, n_kv=n_kv, head_dim=d, dtype=c.ctx.dtype, n_slots=n_slots, k_pools=[pools[0]],
                     v_pools=[pools[1]], hot_fraction=10.5 / n_slots, kv8=True)
    k, v = (c.to(_odd_values(rng, _rows(rng, N, n_kv, d, dtype))).float().cpu().numpy() for _ in range(2))
    slots = (10 + rng.permutation(n_slots - 10)[:N]).astype(np.int32)
    ctx.cold_append(0, c.to(k), c.to(v), torch.from_numpy(slots).cuda(), N)
    ctx.sync_status()
    for pool, x in zip(pools, (k, v)):
        got = pool.cpu().numpy()
        codes, scales = K8.quantise(x, 1)
        live = got[slots]
        assert ((live[:, : n_kv * d].reshape(N, n_kv, d) == codes) | (((codes & 0x7F) == 0x7F) & ((live[:, : n_kv * d].reshape(N, n_kv, d) & 0x7F) == 0x7F))).all()
        assert np.array_equal(live[:, n_kv * d : n_kv * (d + 4)].copy().view(np.float32), scales)
        rest = np.delete(got, slots, axis=0)
        assert (rest == 0xFF).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("slab", [False, True])
def test_write_next_to_halfway_points(cuda_ok, dtype, slab):
    """Elements on, and a few last places beside, the halfway points of two codes, for many scales."""
    torch, gb, rng = _torch(), _gb(), np.random.default_rng(27)
    grid = K8.e4m3_values()[:127]
    mids = np.concatenate([(grid[:-1] + grid[1:]) / 2, [0.0, 2.0 ** -10, 1e-30]])
    amax = np.concatenate([2.0 ** rng.uniform(-90, 100, 150), rng.uniform(0.5, 4.0, 300), [2.0 ** -96, 1.0, 3.3e38, 1.75]])
    if dtype == "bf16":
        amax = torch.from_numpy(amax.astype(np.float32)).to(torch.bfloat16).float().numpy().astype(np.float64)
    amax = amax.astype(np.float32)
    x = (mids[None] * amax[:, None].astype(np.float64) / 448.0).astype(np.float32)
    step = 1 if dtype == "f32" else 1 << 16
    u = (x.view(np.int32)[:, None] // step + rng.integers(-3, 4, (len(amax), 7, 1))) * step  # last places of the type
    x = np.maximum(u, 0).astype(np.int32).view(np.float32).reshape(len(amax), -1)
    x = np.where(np.isfinite(x), np.minimum(x, amax[:, None]), 0.0) * rng.choice([-1.0, 1.0], x.shape)
    n, d, block = len(amax), 256, K8.BLOCK if slab else 1
    heads = np.zeros((n, 4, d), dtype=np.float32)
    heads[:, :, 0] = amax[:, None]
    heads[:, :, 1:] = np.pad(x, ((0, 0), (0, 4 * (d - 1) - x.shape[1]))).reshape(n, 4, d - 1)
    if slab:
        heads[:, :, 0] = 0.0
        heads = np.clip(heads / amax[:, None, None], -1, 1).astype(np.float32) * np.float32(1.6171875)
        heads[::block, :, 0] = 1.6171875
    c = Kv8(rng, n_q=4, n_kv=4, d=d, dtype=dtype)
    heads = c.to(heads).float().cpu().numpy()
    n_slots = n + 40
    pools = [torch.full((n_slots, c.row), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    n_hot = n + 10 if slab else 10
    ctx = gb.Context(n_layers=1, n_q=4, n_kv=4, head_dim=d, dtype=c.ctx.dtype, n_slots=n_slots, k_pools=[pools[0]], v_pools=[pools[1]],
                     hot_fraction=(n_hot + 0.5) / n_slots, kv8=True)
    if slab:
        sid, at = ctx.hot_alloc(n)
        ctx.hot_fill(0, sid, c.to(heads), c.to(heads))
        slots = np.arange(at, at + n)
    else:
        slots = (10 + rng.permutation(n_slots - 10)[:n]).astype(np.int32)
        ctx.cold_append(0, c.to(heads), c.to(heads), torch.from_numpy(slots).cuda(), n)
    ctx.sync_status()
    codes, scales = K8.quantise(heads, block)
    for pool in pools:
        got = pool.cpu().numpy()[slots]
        assert np.array_equal(got[:, : 4 * d].reshape(n, 4, d), codes)
        assert np.array_equal(got[:, 4 * d : 4 * (d + 4)].copy().view(np.float32), scales)


def test_token_write_refuses_bad_slots(cuda_ok):
    torch, gb, rng = _torch(), _gb(), np.random.default_rng(5)
    c = Kv8(rng, n_q=2, n_kv=2, d=64, dtype="bf16", prefixes=[10])
    before = c.kp.clone()
    x = c.to(_rows(rng, 3, 2, 64, "bf16"))
    c.ctx.cold_append(0, x, x, torch.tensor([0, -1, c.kp.shape[0]], dtype=torch.int32, device="cuda"), 3)
    with pytest.raises(gb.DeviceCheckFailed):
        c.ctx.sync_status()
    assert torch.equal(before, c.kp)


# ---- attention --------------------------------------------------------------------------------

HEADS = [(32, 8, 128, "bf16"), (40, 8, 128, "bf16"), (4, 4, 128, "bf16"), (7, 1, 128, "bf16"), (16, 2, 128, "bf16"), (6, 3, 128, "bf16"),
         (24, 2, 128, "bf16"), (8, 2, 64, "f32"), (9, 3, 96, "bf16"), (4, 2, 256, "f32"), (20, 1, 32, "f32"), (10, 10, 128, "bf16")]


@pytest.mark.parametrize("n_q,n_kv,d,dtype", HEADS)
def test_decode_matches_64_bit(cuda_ok, n_q, n_kv, d, dtype):
    """Ragged prefixes with a prefix-less, a prefix-only and a one-token request."""
    rng = np.random.default_rng([n_q, n_kv, d])
    c = Kv8(rng, n_q=n_q, n_kv=n_kv, d=d, dtype=dtype, prefixes=[517, 130], of=[0, 1, -1, 0, 0, 1, 0, -1, 0],
            lens=[5, 33, 70, 0, 1, 16, 200, 17, 64], slots_before=9)
    c.check(*c.decode(), f"{n_q}/{n_kv}/{d}/{dtype}")


@pytest.mark.parametrize("L_p", [1, 15, 63, 64, 65, 127, 128, 129, 300, 1000])
def test_decode_prefix_lengths(cuda_ok, L_p):
    rng = np.random.default_rng(L_p)
    c = Kv8(rng, n_q=32, n_kv=8, d=128, dtype="bf16", prefixes=[L_p], of=[0, 0], lens=[0, 3], slots_before=L_p % 7)
    c.check(*c.decode(), f"L_p {L_p}")


@pytest.mark.parametrize("B", [1, 3, 33, 100])
@pytest.mark.parametrize("n_q", [8, 40, 64])
def test_decode_rows_of_a_group(cuda_ok, B, n_q):
    """From one row a KV head to several row blocks, the group's requests scattered over the batch."""
    rng = np.random.default_rng([B, n_q])
    c = Kv8(rng, n_q=n_q, n_kv=8, d=128, dtype="bf16", prefixes=[390, 64], of=[b * 7 % 3 % 2 for b in range(B)],
            lens=[int(x) for x in rng.integers(0, 20, B)])
    c.check(*c.decode(), f"B {B} n_q {n_q}")


@pytest.mark.parametrize("lens", [[1], [15], [16], [17], [31, 1], [5000], [1, 2, 3, 4, 700, 5], [33] * 50])
def test_decode_cold_lengths(cuda_ok, lens):
    rng = np.random.default_rng(sum(lens))
    c = Kv8(rng, n_q=32, n_kv=8, d=128, dtype="bf16", of=[-1] * len(lens), lens=lens)
    c.check(*c.decode(), f"COLD {lens[:4]}")


def test_decode_peaked_and_uneven_scales(cuda_ok):
    """Scores far apart, and blocks and tokens whose K or V scales differ by many powers of two: a
    sink token with small V, and blocks with large ones."""
    def edit(kind, k, v):
        n = k.shape[0]
        if kind == "prefix":
            v[:64] *= np.float32(2.0 ** -12)
            v[64:128] *= np.float32(2.0 ** 10)
            k[:64] *= np.float32(2.0 ** 3)
            k[128:192] *= np.float32(2.0 ** -20)
        for t in range(0, n, 3):
            v[t] *= np.float32(2.0 ** ((t % 31) - 15))
    rng = np.random.default_rng(11)
    c = Kv8(rng, n_q=32, n_kv=8, d=128, dtype="bf16", prefixes=[700], of=[0, 0, -1], lens=[100, 0, 300], q_scale=2.0, edit=edit)
    c.check(*c.decode(), "uneven")


def test_decode_zero_rows(cuda_ok):
    """All-zero K (equal scores) and all-zero V blocks."""
    def edit(kind, k, v):
        k[:] = 0.0
        v[: k.shape[0] // 2] = 0.0
    rng = np.random.default_rng(12)
    c = Kv8(rng, n_q=16, n_kv=4, d=128, dtype="bf16", prefixes=[200], of=[0, -1], lens=[20, 40], edit=edit)
    c.check(*c.decode(), "zeros")


def test_decode_large_queries(cuda_ok):
    """q beyond fp16's range in some rows (bf16 holds it), tiny in others."""
    rng = np.random.default_rng(13)
    c = Kv8(rng, n_q=8, n_kv=2, d=128, dtype="bf16", prefixes=[150], of=[0, 0, -1], lens=[10, 0, 30], edit=lambda kind, k, v: k.__imul__(np.float32(2.0 ** -17)))
    torch = _torch()
    scale = torch.tensor([2.0 ** 18, 2.0 ** 17, 1.0, 2.0 ** -30, 2.0 ** 16, 0.0, 2.0 ** -3, 2.0 ** 14], device="cuda")[None, :, None]
    c.q = (c.q.float() * scale).to(torch.bfloat16)
    c.q_host = c.q.float().cpu().numpy().astype(np.float64)
    c.check(*c.decode(), "large q")


def test_decode_nan_stays_with_its_head(cuda_ok):
    """A NaN in one head of one token's V reaches that head's output column of the requests that
    attend it, and nothing else."""
    torch, rng = _torch(), np.random.default_rng(14)
    c = Kv8(rng, n_q=16, n_kv=4, d=128, dtype="bf16", prefixes=[100], of=[0, -1, 0], lens=[20, 40, 5])
    o, lse = c.decode()
    k, v = (torch.randn(1, 4, 128, device="cuda").to(torch.bfloat16) for _ in range(2))
    v[0, 2, 7] = float("nan")
    slot = c.table[1, 3:4].contiguous()
    c.ctx.cold_append(0, k, v, slot, 1)
    o2, lse2 = c.decode()
    bad = torch.isnan(o2)
    want = torch.zeros_like(bad)
    want[1, 8:12, 7] = True
    assert torch.equal(bad, want)
    assert torch.equal(o2[[0, 2]], o[[0, 2]]) and torch.equal(lse2[[0, 2]], lse[[0, 2]]) and not torch.isnan(lse2).any()


@pytest.mark.parametrize("n_q,n_kv,d,dtype", [(32, 8, 128, "bf16"), (8, 2, 64, "f32"), (6, 3, 128, "bf16")])
@pytest.mark.parametrize("on_device", [False, True])
def test_fused_append_equals_append_then_decode(cuda_ok, n_q, n_kv, d, dtype, on_device):
    torch, gb, rng = _torch(), _gb(), np.random.default_rng(15)
    lens = [1, 16, 17, 40]
    c = Kv8(rng, n_q=n_q, n_kv=n_kv, d=d, dtype=dtype, prefixes=[70], of=[0, 0, -1, 0], lens=lens)
    k, v = (c.to(_rows(rng, 4, n_kv, d, dtype)) for _ in range(2))
    batch = gb.Batch([c.slabs[i] if i >= 0 else -1 for i in c.of], [n + 3 for n in lens], c.table, c.cap, c.live) if on_device else c.batch
    o1, lse1 = c.decode(batch=batch, k_new=k, v_new=v)
    pools = c.kp.clone(), c.vp.clone()
    newest = torch.stack([c.table[b, n - 1] for b, n in enumerate(lens)])
    c.kp[newest.long()] = 0xFF
    c.vp[newest.long()] = 0xFF
    c.ctx.cold_append(0, k, v, newest, 4)
    o2, lse2 = c.decode(batch=batch)
    assert torch.equal(o1, o2) and torch.equal(lse1, lse2)
    assert torch.equal(pools[0], c.kp) and torch.equal(pools[1], c.vp)
    for b, n in enumerate(lens):
        c.ck[b][n - 1] = K8.through_cache(k[b:b + 1].float().cpu().numpy(), 1)[0]
        c.cv[b][n - 1] = K8.through_cache(v[b:b + 1].float().cpu().numpy(), 1)[0]
    c.check(o1, lse1, "append")


def test_decode_in_a_graph_on_another_stream(cuda_ok):
    """Captured once and replayed with new q, growing live lengths and new slots' contents; two
    graphs share one workspace and replay in turn."""
    torch, gb, rng = _torch(), _gb(), np.random.default_rng(16)
    lens = [30, 9, 64]
    c = Kv8(rng, n_q=32, n_kv=8, d=128, dtype="bf16", prefixes=[200], of=[0, -1, 0], lens=lens)
    batch = gb.Batch([c.slabs[i] if i >= 0 else -1 for i in c.of], lens, c.table, c.cap, c.live)
    plan = c.ctx.dispatch(batch)
    ws = torch.empty(c.ctx.workspace_size(plan), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.ctx.decode_attention(0, c.q, batch, plan, o, lse, ws, ws.numel(), s)
    s.synchronize()
    graphs = []
    outs = []
    for _ in range(2):
        og, lg = torch.empty_like(o), torch.empty_like(lse)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.ctx.decode_attention(0, c.q, batch, plan, og, lg, ws, ws.numel(), s)
        graphs.append(g)
        outs.append((og, lg))
    full_k, full_v = list(c.ck), list(c.cv)
    for live in ([30, 9, 64], [7, 1, 16], [29, 9, 0]):
        c.live.copy_(torch.tensor(live, dtype=torch.int32))
        q = torch.randn_like(c.q)
        c.q.copy_(q)
        c.q_host = q.double().cpu().numpy()
        torch.cuda.synchronize()
        for g in graphs:
            with torch.cuda.stream(s):
                g.replay()
        s.synchronize()
        c.lens, c.ck, c.cv = live, [k[:n] for k, n in zip(full_k, live)], [v[:n] for v, n in zip(full_v, live)]
        for og, lg in outs:
            c.check(og, lg, f"replay {live}")
    c.ctx.sync_status()


def test_decode_far_slots(cuda_ok):
    """Slots whose byte offsets pass 2^32, in slab and COLD pool."""
    torch, gb, rng = _torch(), _gb(), np.random.default_rng(17)
    n_kv, d, n_q = 8, 128, 32
    row = gb.kv8_row_bytes(n_kv, d)
    n_slots = 2 ** 33 // row + 4000
    kp, vp = (torch.zeros((n_slots, row), dtype=torch.uint8, device="cuda") for _ in range(2))
    n_hot = n_slots - 2000
    ctx = gb.Context(n_layers=1, n_q=n_q, n_kv=n_kv, head_dim=d, dtype=gb.DTYPE_BF16, n_slots=n_slots, k_pools=[kp], v_pools=[vp],
                     hot_fraction=(n_hot + 0.5) / n_slots, kv8=True, max_batch=4)
    ctx.hot_alloc(n_hot - 300)
    sid, off = ctx.hot_alloc(300)
    assert off * row > 2 ** 32
    c = Kv8(rng, n_q=n_q, n_kv=n_kv, d=d, dtype="bf16", prefixes=[300], of=[0, -1], lens=[40, 60])
    ctx.hot_fill(0, sid, c.to(c.pk[0].astype(np.float32)), c.to(c.pv[0].astype(np.float32)))
    # what that wrote is the quantised quantised rows; read the pool back for the reference
    table = torch.full((2, 64), -1, dtype=torch.int32, device="cuda")
    table[0, :40] = torch.arange(n_slots - 40, n_slots, device="cuda")
    table[1, :60] = torch.arange(n_slots - 200, n_slots - 140, device="cuda").flip(0)
    for b, n in enumerate([40, 60]):
        ctx.cold_append(0, c.to(c.ck[b].astype(np.float32)), c.to(c.cv[b].astype(np.float32)), table[b, :n].contiguous(), n)

    def read(pool, slots):
        rows = pool[slots.long()].cpu().numpy()
        return K8.values(rows[:, : n_kv * d].reshape(-1, n_kv, d), rows[:, n_kv * d : n_kv * (d + 4)].copy().view(np.float32))

    hot = torch.arange(off, off + 300, device="cuda")
    c.pk, c.pv = [read(kp, hot)], [read(vp, hot)]
    c.ck, c.cv = ([read(pool, table[b, :n]) for b, n in enumerate([40, 60])] for pool in (kp, vp))
    c.ctx, c.batch = ctx, gb.Batch([sid, -1], [40, 60], table, 64)
    c.check(*c.decode(), "far slots")


def test_decode_bad_slot_is_latched(cuda_ok):
    gb, rng = _gb(), np.random.default_rng(18)
    c = Kv8(rng, n_q=32, n_kv=8, d=128, dtype="bf16", of=[-1, -1], lens=[40, 20])
    c.table[0, 7] = c.kp.shape[0] + 5
    with pytest.raises(gb.DeviceCheckFailed):
        c.decode()
    c.table[0, 7] = -3
    with pytest.raises(gb.DeviceCheckFailed):
        c.decode()


def test_stalled_wait_is_reported_and_the_context_survives(cuda_ok):
    gb, rng = _gb(), np.random.default_rng(30)
    c = Kv8(rng, n_q=32, n_kv=8, d=128, dtype="bf16", prefixes=[300], of=[0, 0, -1], lens=[40, 20, 70])
    c.check(*c.decode(), "before")
    c.ctx.inject_stall(True)
    with pytest.raises(gb.DeviceCheckFailed):
        c.decode()
    c.check(*c.decode(), "after")


def test_prefill_is_refused_and_static_workspace_serves(cuda_ok):
    torch, gb, rng = _torch(), _gb(), np.random.default_rng(19)
    c = Kv8(rng, n_q=32, n_kv=8, d=128, dtype="bf16", prefixes=[100], of=[0], lens=[20])
    q = torch.zeros(100, 32, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    with pytest.raises(gb.GranikvError) as e:
        c.ctx.prefill_attention(0, c.slabs[0], None, None, q, q, torch.empty(100, 32, device="cuda"), ws, ws.numel())
    assert e.value.status == gb.ERR_UNSUPPORTED
    o, lse = c.decode()
    plan = c.ctx.dispatch(c.batch)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    c.ctx.decode_attention_static(0, c.q, c.batch, plan, o2, lse2)
    c.ctx.sync_status()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_backends_agree(cuda_ok):
    gb = _gb()
    for backend in (gb.BACKEND_DENSE, gb.BACKEND_CASCADE):
        c = Kv8(np.random.default_rng(20), n_q=32, n_kv=8, d=128, dtype="bf16", prefixes=[333], of=[0, 0, 0], lens=[12, 0, 50], backend=backend)
        c.check(*c.decode(), f"backend {backend}")


SCHEDULES = {"serial": lambda x: x.set_concurrency(False), "half": lambda x: x.set_concurrency(True, 0.5),
             "all": lambda x: x.set_concurrency(True, 1.0), "ahead": lambda x: x.set_dense_l2_ahead(4),
             "unfused": lambda x: x.set_fused_merge(False), "fused": lambda x: x.set_fused_merge(True),
             "mixed": lambda x: x.set_msat(30), "cascade": lambda x: x.set_msat(10000)}


@pytest.mark.parametrize("how", sorted(SCHEDULES))
def test_decode_schedules(cuda_ok, how):
    """Every knob of the schedule leaves the result within the same tolerance; `mixed` runs one group
    on the tensor cores and one on CUDA cores."""
    rng = np.random.default_rng(22)
    c = Kv8(rng, n_q=32, n_kv=8, d=128, dtype="bf16", prefixes=[1500, 700], of=[0, 1, 0, 0, -1, 0, 0, 0, 0, 0], lens=[300, 20, 0, 1, 90, 64, 700, 33, 5, 16])
    SCHEDULES[how](c.ctx)
    c.check(*c.decode(), how)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("backend", ["dense", "cascade"])
def test_decode_bad_query_stays_with_its_head(cuda_ok, bad, backend):
    """A NaN or infinity in one head's q makes that head's row NaN and changes no other."""
    torch, gb, rng = _torch(), _gb(), np.random.default_rng(23)
    c = Kv8(rng, n_q=32, n_kv=8, d=128, dtype="bf16", prefixes=[300], of=[0, 0, -1], lens=[20, 0, 70],
            backend=gb.BACKEND_DENSE if backend == "dense" else gb.BACKEND_CASCADE)
    o, lse = c.decode()
    for b, h in ((0, 5), (1, 31), (2, 0)):
        c.q[b, h, 77] = bad
    o2, lse2 = c.decode()
    hit = torch.zeros_like(lse, dtype=torch.bool)
    hit[0, 5] = hit[1, 31] = hit[2, 0] = True
    assert torch.equal(torch.isnan(o2).any(dim=2), hit) and torch.isnan(o2[hit]).all() and torch.equal(torch.isnan(lse2), hit)
    assert torch.equal(o2[~hit], o[~hit]) and torch.equal(lse2[~hit], lse[~hit])


@pytest.mark.parametrize("shape", [(32, 8, 128, "bf16"), (8, 2, 64, "f32")])
@pytest.mark.parametrize("where", ["prefix", "cold"])
def test_decode_nan_key_reaches_its_readers(cuda_ok, shape, where):
    """A NaN in one head of one token's K makes that head NaN for the requests that attend the token."""
    torch = _torch()
    n_q, n_kv, d, dtype = shape

    def case(edit):
        return Kv8(np.random.default_rng(26), n_q=n_q, n_kv=n_kv, d=d, dtype=dtype, prefixes=[300], of=[0, -1, 0], lens=[20, 40, 0], edit=edit)

    def edit(kind, k, v):
        if kind == where and k.shape[0] in (300, 40):
            k[17, 1, 9] = np.nan

    (o, lse), (o2, lse2) = (case(e).decode() for e in (None, edit))
    g = n_q // n_kv
    hit = torch.zeros_like(lse, dtype=torch.bool)
    hit[[0, 2] if where == "prefix" else [1], g:2 * g] = True
    assert torch.equal(torch.isnan(lse2), hit) and torch.isnan(o2[hit]).all()
    assert torch.equal(o2[~hit], o[~hit]) and torch.equal(lse2[~hit], lse[~hit])


def test_decode_on_two_streams_at_once(cuda_ok):
    """One plan, two workspaces, two streams: the results of the calls one after the other."""
    torch, rng = _torch(), np.random.default_rng(24)
    c = Kv8(rng, n_q=32, n_kv=8, d=128, dtype="bf16", prefixes=[2000], of=[0] * 8 + [-1], lens=[int(x) for x in rng.integers(0, 400, 8)] + [40])
    o, lse = c.decode()
    plan = c.ctx.dispatch(c.batch)
    n = c.ctx.workspace_size(plan)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.empty_like(o), torch.empty_like(lse), torch.empty(n, dtype=torch.uint8, device="cuda")) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (a, b, ws) in zip(streams, outs):
            c.ctx.decode_attention(0, c.q, c.batch, plan, a, b, ws, n, s)
    torch.cuda.synchronize()
    c.ctx.sync_status()
    for a, b, _ in outs:
        assert torch.equal(a, o) and torch.equal(b, lse)


def test_decode_the_same_slot_twice(cuda_ok):
    """A slot named twice in a row, and by two rows, counts once for each place."""
    rng = np.random.default_rng(25)
    c = Kv8(rng, n_q=32, n_kv=8, d=128, dtype="bf16", prefixes=[90], of=[0, -1, 0], lens=[40, 35, 7])
    c.table[0, 3], c.table[0, 39], c.table[2, 6] = c.table[0, 4], c.table[0, 4], c.table[1, 20]
    for x in (c.ck, c.cv):
        x[0][3] = x[0][39] = x[0][4]
        x[2][6] = x[1][20]
    c.check(*c.decode(), "twice")


def test_cache_in_8_bits_with_prefix_lifecycle(cuda_ok):
    """GraniKVCache(kv8=True): admission to HOT, fallback to COLD shared by two requests, appends,
    decode with the newest token written by the call."""
    torch, gb = _torch(), _gb()
    from shared_prefix_kv_decode_gb300 import GraniKVCache
    rng = np.random.default_rng(21)
    cache = GraniKVCache(n_layers=1, n_q=32, n_kv=8, head_dim=128, dtype=gb.DTYPE_BF16, n_slots=2000, max_batch=4, cap=400, kv8=True)
    assert cache.k_pools[0].dtype == torch.uint8
    c = Kv8(rng, n_q=32, n_kv=8, d=128, dtype="bf16")  # draws and checks
    lens = [300, 250]
    ks, vs = ([_rows(rng, n, 8, 128, "bf16") for n in lens] for _ in range(2))
    toks = [[1] * 300, [2] * 250]
    infos, slabs = [], []
    for i, rows in enumerate(((0,), (1, 2))):  # the first prefix is referenced before the second comes, so it stays in HOT
        infos.append(cache.admit(toks[i], [c.to(ks[i])], [c.to(vs[i])])[0])
        slabs += [cache.attach(b, toks[i] + [9])[0] for b in rows]
    assert infos[0]["slab_id"] >= 0 and infos[1]["slab_id"] == -1
    own = [5, 17, 0]
    kn, vn = (_rows(rng, sum(own) + 3, 8, 128, "bf16") for _ in range(2))
    cache.append(own, [c.to(kn[: sum(own)])], [c.to(vn[: sum(own)])])
    cache.alloc([1, 1, 1])
    batch = cache.batch(slabs + [], cache.seq_len_host[:3])
    q = torch.randn(3, 32, 128, device="cuda").to(torch.bfloat16)
    o, lse = cache.decode(0, q, batch, k_new=c.to(kn[-3:]), v_new=c.to(vn[-3:]))
    cache.ctx.sync_status(cache.stream())
    tk, tv = K8.through_cache(kn, 1), K8.through_cache(vn, 1)
    pk = [K8.through_cache(ks[0], 64), K8.through_cache(ks[1], 1)]
    pv = [K8.through_cache(vs[0], 64), K8.through_cache(vs[1], 1)]
    at = np.cumsum([0] + own)
    c.of, c.lens = [-1] * 3, [1] * 3
    c.ck = [np.concatenate([pk[min(b, 1)], tk[at[b]:at[b + 1]], tk[len(tk) - 3 + b][None]]) for b in range(3)]
    c.cv = [np.concatenate([pv[min(b, 1)], tv[at[b]:at[b + 1]], tv[len(tv) - 3 + b][None]]) for b in range(3)]
    c.q_host = q.double().cpu().numpy()
    c.check(o, lse, "cache")


@pytest.mark.parametrize("n_q,n_kv,d,dtype", [(32, 8, 128, "bf16"), (24, 2, 128, "bf16"), (9, 3, 96, "bf16"), (8, 2, 64, "f32")])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf")])
@pytest.mark.parametrize("backend", ["dense", "cascade"])
def test_decode_infinite_query_over_keys_of_one_sign(cuda_ok, n_q, n_kv, d, dtype, bad, backend):
    """Every K has the same sign in the dimension where q is infinite, so all scores of the head are -inf
    (or all +inf): its row is NaN all the same, with and without a slab, down to one token."""
    torch, gb = _torch(), _gb()

    def edit(kind, k, v):
        k[:, :, 7] = -np.abs(k[:, :, 7]) - 1.0

    c = Kv8(np.random.default_rng([n_q, d]), n_q=n_q, n_kv=n_kv, d=d, dtype=dtype, prefixes=[150], of=[0, -1, -1, 0], lens=[20, 1, 70, 0],
            edit=edit, backend=gb.BACKEND_DENSE if backend == "dense" else gb.BACKEND_CASCADE)
    o, lse = c.decode()
    hit = torch.zeros_like(lse, dtype=torch.bool)
    for b, h in ((0, 1), (1, 0), (2, n_q - 1), (3, 2)):
        c.q[b, h, 7] = bad
        hit[b, h] = True
    o2, lse2 = c.decode()
    assert torch.equal(torch.isnan(lse2), hit) and torch.isnan(o2[hit]).all()
    assert torch.equal(o2[~hit], o[~hit]) and torch.equal(lse2[~hit], lse[~hit])


def test_decode_long_cold_runs_of_zero_values(cuda_ok):
    """More than 600 COLD tokens of equal weight in one run, their V all zero: o is 0 (or the prefix's share)
    and lse finite.  The prefix side takes all SMs but two, so the 3,000 tokens make two runs."""
    def edit(kind, k, v):
        if kind == "cold":
            k[:] = 0.0
            v[:] = 0.0
    c = Kv8(np.random.default_rng(31), n_q=4, n_kv=1, d=128, dtype="bf16", prefixes=[19200], of=[0, -1], lens=[1500, 1500], edit=edit)
    c.ctx.set_concurrency(True, 0.99)
    plan = c.ctx.dispatch(c.batch)
    assert sum(c.lens) > 600 * plan.suffix_runs()["runs"]
    o, lse = c.decode(plan)
    assert not o[1].any()
    c.check(o, lse, "zero V")


def _uneven_v(e, small, where, of):
    """V of about 2^e, and of `small` 2^-e or nothing in some blocks of a slab or COLD tokens."""
    def edit(kind, k, v):
        if kind != of and of != "both":
            return
        n, step = k.shape[0], K8.BLOCK if kind == "prefix" else 1
        at = np.arange(n) // step
        low = {"first": at <= at[-1] // 2, "last": at > at[-1] // 2, "alternate": at % 2 == 1}[where] if n else np.zeros(0, bool)
        v[~low] *= np.float32(2.0 ** e)
        v[low] *= np.float32(small * 2.0 ** -e)
        k[low] *= np.float32(2.0)
    return edit


UNEVEN = [(32, 8, 128, "bf16"), (16, 2, 128, "bf16"), (24, 2, 128, "bf16"), (8, 2, 64, "f32")]


@pytest.mark.parametrize("n_q,n_kv,d,dtype", UNEVEN)
@pytest.mark.parametrize("e", [20, 62, 100])
@pytest.mark.parametrize("small", [0.0, 1.0])
@pytest.mark.parametrize("where", ["first", "last", "alternate"])
def test_decode_cold_values_far_apart(cuda_ok, n_q, n_kv, d, dtype, e, small, where):
    """A COLD token keeps its weight in o and lse however small its V is beside the others'."""
    c = Kv8(np.random.default_rng([e, n_q]), n_q=n_q, n_kv=n_kv, d=d, dtype=dtype, prefixes=[90], of=[-1, -1, -1, 0], lens=[100, 2, 300, 40],
            edit=_uneven_v(e, small, where, "cold"))
    c.check(*c.decode(), f"{e} {small} {where}")


@pytest.mark.parametrize("n_q,n_kv,d,dtype", UNEVEN)
@pytest.mark.parametrize("e", [20, 62, 100])
@pytest.mark.parametrize("small", [0.0, 1.0])
@pytest.mark.parametrize("where", ["first", "last", "alternate"])
def test_decode_prefix_values_far_apart(cuda_ok, n_q, n_kv, d, dtype, e, small, where):
    """A slab's token keeps its weight in o and lse however small its block's V is beside the others'; pieces of
    one tile to many."""
    c = Kv8(np.random.default_rng([e, n_q, 1]), n_q=n_q, n_kv=n_kv, d=d, dtype=dtype, prefixes=[1100, 300], of=[0, 1, 0, 1], lens=[0, 3, 20, 0],
            edit=_uneven_v(e, small, where, "prefix"))
    c.check(*c.decode(), f"{e} {small} {where}")


def test_decode_long_prefix_pieces_of_zero_values(cuda_ok):
    """A piece of 1,064 tokens whose V is all zero and whose first block scores 2^7.65 below the rest, which the
    kernel's running maximum does not follow: o is 0 and lse finite.  160 requests make 80 CTAs, so that the
    prefix is one piece.  lse: a score of 128 equal products errs by 128 2^-24 of itself, the sum by L 2^-24, the
    exponential and logarithm by 2^-20, lse by 2^-23 of itself."""
    torch = _torch()

    def edit(kind, k, v):
        k[:64], k[64:] = 0.0, 0.46875
        v[:] = 0.0
    c = Kv8(np.random.default_rng(32), n_q=64, n_kv=8, d=128, dtype="bf16", prefixes=[1064], of=[0] * 160, lens=[0] * 160, edit=edit)
    c.q.fill_(1.0)
    plan = c.ctx.dispatch(c.batch)
    assert plan.groups()[0]["n_splits"] == 1
    o, lse = c.decode(plan)
    assert not o.any()
    s = 0.46875 * math.sqrt(128)
    want = math.log(64 + 1000 * math.exp(s))
    assert (lse.double() - want).abs().max().item() <= 128 * 2.0 ** -24 * s + 1064 * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * want


def test_decode_long_pieces_of_values_far_apart(cuda_ok):
    """A piece of more than 132 blocks (160 requests of 64 heads make 80 row blocks), V zero but for blocks 129 to
    131 of about 2^60, K zero: every weight is 1 / 17,000.  Tolerance of o as at the top, all weights equal."""
    L = 17000

    def edit(kind, k, v):
        k[:] = 0.0
        v *= np.float32(2.0 ** 60)
        v[:129 * 64] = 0.0
        v[132 * 64:] = 0.0
    c = Kv8(np.random.default_rng(34), n_q=64, n_kv=1, d=128, dtype="bf16", prefixes=[L], of=[0] * 160, lens=[0] * 160, edit=edit)
    plan = c.ctx.dispatch(c.batch)
    assert plan.groups()[0]["n_splits"] <= 2
    o, lse = c.decode(plan)
    V = c.pv[0][:, 0]
    want, A = V.sum(axis=0) / L, np.abs(V).sum(axis=0) / L
    tol = (L * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -11) * A + 2.0 ** -32 * np.abs(V).max()
    tol += 2.0 ** -8 * (np.abs(want) + tol)
    o = o.double().cpu().numpy().reshape(-1, 128)
    assert (np.abs(o - want) <= tol).all()
    assert (lse.double() - math.log(L)).abs().max().item() <= L * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * math.log(L)


@pytest.mark.parametrize("L_p", [1, 70, 200])
@pytest.mark.parametrize("size", [2.0 ** -30, 2.0 ** -40, 2.0 ** -100])
def test_decode_tiny_queries_over_zero_keys(cuda_ok, L_p, size):
    """All-zero K and a q so small that the product of the scales underflows: the weights are equal, the places
    past the prefix's end still have none."""
    def edit(kind, k, v):
        k[:] = 0.0
    c = Kv8(np.random.default_rng(33), n_q=32, n_kv=8, d=128, dtype="bf16", prefixes=[L_p], of=[0, 0, -1], lens=[0, 5, 9], q_scale=size, edit=edit)
    c.check(*c.decode(), f"{L_p} {size}")


@pytest.mark.parametrize("n_q,n_kv", [(8, 2), (32, 8), (12, 1), (24, 12)])
def test_decode_bf16_heads_of_64(cuda_ok, n_q, n_kv):
    rng = np.random.default_rng([n_q, n_kv, 64])
    c = Kv8(rng, n_q=n_q, n_kv=n_kv, d=64, dtype="bf16", prefixes=[517, 130], of=[0, 1, -1, 0, 0, 1, 0, -1, 0],
            lens=[5, 33, 70, 0, 1, 16, 200, 17, 64], slots_before=9)
    c.check(*c.decode(), f"{n_q}/{n_kv}/64/bf16")
