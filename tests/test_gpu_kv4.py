"""The 4-bit cache on the GPU: what the writes put into the pools, bit for bit; what reading back gives,
exactly; decode attention and the weights of COLD tokens over it against 64 bits on the values held.

Every pool starts as 0xff bytes (NaN scales, infinite exponents), so anything read outside the written slots
poisons the result.

Tolerances.  With A = sum_t p_t |v_t| (64 bits) over a row's L keys:
  o:   the weights are rounded to fp16 at most (half a step: 2^-11 relative), products and sums are
       fp32, whose error over L terms is at most L 2^-24 relative to A, the normalisation and merge
       add a few 2^-24; an error of x in a score moves its weight by x relative (below).  The result
       is rounded to bf16 (2^-8 relative to it) or kept in fp32.  An fp16 weight P = 2^7 p u / M, with u the
       token's power of two for V and M = max_t p_t u_t (the kernel may carry more than 2^7, never less), that falls
       below 2^-14 is off by at most half of fp16's last subnormal, 2^-25: by 2^-32 M in p u, which meets
       a code times scale of at most 2688: 2^-32 max_t(p_t 2688 u_t) for each of the L tokens.
  lse: a score q.k is a sum of d exact products in fp32: error x of at most d 2^-24 sum|q_i k_i| scale; q
       in fp16 is exact but for elements 2^-31 below its row's largest, which are off by 2^-39 of that at
       most: 2^-39 max|q| sum|k_i| scale more;
       the exponential and logarithm add 2^-20, the sum of L weights L 2^-24.
fp32 contexts keep the weights in fp32, and so have no 2^-11."""

import math

import numpy as np
import pytest

import oracle.kv4 as K4
import oracle.kv8 as K8
from tests.test_gpu_kv8 import _gb, _odd_values, _rows, _torch

pytestmark = pytest.mark.gpu

BLOCK = K4.BLOCK


class Kv4:
    """A 4-bit context with poisoned pools, its prefixes in slabs and its COLD rows at scattered slots."""

    def __init__(self, rng, *, n_q, n_kv, d, dtype, prefixes=(), of=(), lens=(), cap=None, slots_before=0,
                 spread=0.5, q_scale=None, holes=7, backend=None, edit=None):
        torch, gb = _torch(), _gb()
        self.n_q, self.n_kv, self.d, self.dtype = n_q, n_kv, d, dtype
        self.tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.prefixes, self.of, self.lens = list(prefixes), list(of), list(lens)
        B = len(self.lens)
        n_cold = sum(lens) + holes
        n_hot = slots_before + sum(prefixes) + holes
        n_slots = n_hot + n_cold
        self.row = gb.kv4_row_bytes(n_kv, d)
        self.kp, self.vp = (torch.full((n_slots, self.row), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.ctx = gb.Context(n_layers=1, n_q=n_q, n_kv=n_kv, head_dim=d, dtype=gb.DTYPE_BF16 if dtype == "bf16" else gb.DTYPE_F32,
                              n_slots=n_slots, k_pools=[self.kp], v_pools=[self.vp], hot_fraction=(n_hot + 0.5) / n_slots,
                              max_batch=max(B, 1), kv4=True)
        if backend is not None:
            self.ctx.force_backend(backend)
        if slots_before:
            self.ctx.hot_alloc(slots_before)
        self.dev = self.kp.device
        self.slabs, self.pk, self.pv, self.pu = [], [], [], []
        for L in self.prefixes:
            k, v = _rows(rng, L, n_kv, d, dtype, spread), _rows(rng, L, n_kv, d, dtype, spread)
            if edit:
                edit("prefix", k, v)
            sid, _ = self.ctx.hot_alloc(L)
            self.ctx.hot_fill(0, sid, self.to(k), self.to(v))
            self.slabs.append(sid)
            self.pk.append(K4.through_cache(k, BLOCK))
            self.pv.append(K4.through_cache(v, BLOCK))
            self.pu.append(K4.units(v, BLOCK))
        self.n_hot = n_hot
        slots = n_hot + rng.permutation(n_cold)[: sum(lens)].astype(np.int32)
        self.cap = cap or max([1] + [n + 3 for n in lens])
        table = np.full((B, self.cap), -1, dtype=np.int32)
        self.ck, self.cv, self.cu, at = [], [], [], 0
        for b, n in enumerate(self.lens):
            table[b, :n] = slots[at:at + n]
            at += n
            k, v = _rows(rng, n, n_kv, d, dtype, spread), _rows(rng, n, n_kv, d, dtype, spread)
            if edit:
                edit("cold", k, v)
            if n:
                self.ctx.cold_append(0, self.to(k), self.to(v), torch.from_numpy(table[b, :n].copy()).to(self.dev), n)
            self.ck.append(K4.through_cache(k, 1))
            self.cv.append(K4.through_cache(v, 1))
            self.cu.append(K4.units(v, 1))
        self.table = torch.from_numpy(table).to(self.dev)
        self.live = torch.tensor(self.lens, dtype=torch.int32, device=self.dev)
        self.batch = gb.Batch([self.slabs[i] if i >= 0 else -1 for i in self.of], self.lens, self.table, self.cap)
        q = torch.from_numpy((rng.standard_normal((B, n_q, d)) * (q_scale or 1.0)).astype(np.float32)).to(self.tdt)
        self.q_host = q.float().numpy().astype(np.float64)
        self.q = q.to(self.dev)

    def to(self, x):
        return _torch().from_numpy(x).to(self.dev).to(self.tdt)

    def set_newest(self, b, k, v):
        """Request b's last COLD token holds the rows k, v (float32 [n_kv, d])."""
        self.ck[b][-1], self.cv[b][-1], self.cu[b][-1] = K4.through_cache(k[None], 1)[0], K4.through_cache(v[None], 1)[0], K4.units(v[None], 1)[0]

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
        parts = [self.ck[b]], [self.cv[b]], [self.cu[b]]
        if self.of[b] >= 0:
            for part, prefix in zip(parts, (self.pk, self.pv, self.pu)):
                part.insert(0, prefix[self.of[b]])
        return [np.concatenate(part) for part in parts]

    def check(self, o, lse, what=""):
        o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
        g = self.n_q // self.n_kv
        for b in range(len(self.lens)):
            K, V, U = self.keys(b)
            L = K.shape[0]
            q = self.q_host[b].reshape(self.n_kv, g, self.d)
            s = np.einsum("jgd,ljd->jgl", q, K) / math.sqrt(self.d)
            x = self.d * 2.0 ** -24 * (np.einsum("jgd,ljd->jgl", np.abs(q), np.abs(K)) / math.sqrt(self.d)).max(axis=2)
            x = x + 2.0 ** -39 * np.abs(q).max(axis=2) * np.abs(K).sum(axis=2).max(axis=0)[:, None] / math.sqrt(self.d)
            m = s.max(axis=2, keepdims=True)
            p = np.exp(s - m)
            ref_lse = (m[..., 0] + np.log(p.sum(axis=2))).reshape(self.n_q)
            p /= p.sum(axis=2, keepdims=True)
            ref = np.einsum("jgl,ljd->jgd", p, V)
            A = np.einsum("jgl,ljd->jgd", p, np.abs(V))
            floor = 2.0 ** -32 * L * (p * 2688.0 * U.T[:, None]).max(axis=2)[..., None] if self.dtype == "bf16" else 0.0
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


def _same_bytes(rows, x, block, n_kv, d):
    """The packed rows hold x: codes, scales and exponents bit for bit (but for the codes beside a NaN), padding untouched."""
    codes, scale, e = K4.unpack_rows(rows, n_kv, d)
    want = K4.quantise(x, block)
    assert np.array_equal(scale, want[1]) and np.array_equal(e, want[2])
    live = np.repeat(want[1] != 0x7F, K4.GROUP, axis=2)
    assert np.array_equal(codes[live], want[0][live])
    assert (rows[:, K4.padding(n_kv, d)] == 0xFF).all()


# ---- writes and reads --------------------------------------------------------------------------

SHAPES = [(8, 128, "bf16"), (2, 64, "f32"), (1, 32, "bf16"), (3, 96, "f32"), (5, 160, "bf16"), (2, 256, "f32"), (4, 192, "bf16"), (1, 224, "f32"),
          (16, 128, "bf16"), (9, 128, "f32")]


def _pools(n_slots, n_kv, d, dtype, n_hot, kind="kv4"):
    """A context of one layer over poisoned pools, and the pools."""
    torch, gb = _torch(), _gb()
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    if kind == "plain":
        pools = [torch.full((n_slots, n_kv, d), float("nan"), dtype=tdt, device="cuda") for _ in range(2)]
    else:
        row = (gb.kv4_row_bytes if kind == "kv4" else gb.kv8_row_bytes)(n_kv, d)
        pools = [torch.full((n_slots, row), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    ctx = gb.Context(n_layers=1, n_q=n_kv, n_kv=n_kv, head_dim=d, dtype=gb.DTYPE_BF16 if dtype == "bf16" else gb.DTYPE_F32, n_slots=n_slots,
                     k_pools=[pools[0]], v_pools=[pools[1]], hot_fraction=(n_hot + 0.5) / n_slots, kv4=kind == "kv4", kv8=kind == "kv8")
    return ctx, pools, tdt


@pytest.mark.parametrize("n_kv,d,dtype", SHAPES)
@pytest.mark.parametrize("L", [1, 63, 64, 65, 200])
def test_slab_write_is_bit_exact(cuda_ok, n_kv, d, dtype, L):
    torch, rng = _torch(), np.random.default_rng([L, n_kv, d])
    ctx, pools, tdt = _pools(L + 40, n_kv, d, dtype, L + 20)
    k, v = (torch.from_numpy(_odd_values(rng, _rows(rng, L, n_kv, d, dtype))).cuda().to(tdt) for _ in range(2))
    ctx.hot_alloc(13)
    sid, off = ctx.hot_alloc(L)
    ctx.hot_fill(0, sid, k, v)
    ctx.sync_status()
    for pool, x in zip(pools, (k, v)):
        got = pool.cpu().numpy()
        _same_bytes(got[off:off + L], x.float().cpu().numpy(), BLOCK, n_kv, d)
        assert (np.concatenate([got[:off], got[off + L:]]) == 0xFF).all()


@pytest.mark.parametrize("n_kv,d,dtype", SHAPES)
@pytest.mark.parametrize("N", [1, 3, 75])
def test_token_write_is_bit_exact(cuda_ok, n_kv, d, dtype, N):
    torch, rng = _torch(), np.random.default_rng([N, n_kv, d])
    n_slots = 2 * N + 30
    ctx, pools, tdt = _pools(n_slots, n_kv, d, dtype, 10)
    k, v = (torch.from_numpy(_odd_values(rng, _rows(rng, N, n_kv, d, dtype))).cuda().to(tdt) for _ in range(2))
    slots = (10 + rng.permutation(n_slots - 10)[:N]).astype(np.int32)
    ctx.cold_append(0, k, v, torch.from_numpy(slots).cuda(), N)
    ctx.sync_status()
    for pool, x in zip(pools, (k, v)):
        got = pool.cpu().numpy()
        _same_bytes(got[slots], x.float().cpu().numpy(), 1, n_kv, d)
        assert (np.delete(got, slots, axis=0) == 0xFF).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("slab", [False, True])
def test_write_at_halfway_points(cuda_ok, dtype, slab):
    """Elements at, and a unit in the last place around, the halfway points of codes under every scale; group maxima
    at and around those of scales."""
    torch, rng = _torch(), np.random.default_rng([slab, dtype == "f32"])
    scales = K8.e4m3_values()[1:127]
    mids = (K4.E2M1[:-1] + K4.E2M1[1:]) / 2
    n_kv, d = 4, 128
    step = 1 if dtype == "f32" else 1 << 16

    def nudge(x):
        u = np.ascontiguousarray(x, dtype=np.float32).view(np.int32).astype(np.int64)
        u = (u // step + rng.integers(-2, 3, u.shape)) * step
        return np.maximum(u, 0).astype(np.int32).view(np.float32)

    rows = []
    for b in scales:  # a group whose largest element gives scale b, the others at b times the halfway points
        for unit in 2.0 ** np.array([0, 3, -20]):
            group = np.empty((4, 16), dtype=np.float32)
            group[:, :14] = nudge(np.tile(np.concatenate([mids, mids]) * b * unit, (4, 1)))
            group[:, 14:] = 6 * b * unit
            rows.append(np.where(rng.random((4, 16)) < 0.5, -group, group))
    for lo, hi in zip(scales[:-1], scales[1:]):  # group maxima around the halfway points of scales
        group = np.zeros((4, 16), dtype=np.float32)
        group[:, 0] = nudge(np.full(4, 6 * (lo + hi) / 2))
        rows.append(group)
    groups = np.concatenate(rows)  # [n, 16]; each goes into a head whose first element holds the unit
    n = len(groups)
    x = np.zeros((n, n_kv, d), dtype=np.float32)
    x[np.arange(n), np.arange(n) % n_kv, 16:32] = groups
    x[:, :, 0] = np.where(np.abs(x).max(axis=2) > 0, 2688.0 * np.exp2(np.ceil(np.log2(np.maximum(np.abs(x).max(axis=2), 1e-30) / 2688))), 0.0)
    if slab:
        x = x[np.argsort(x[:, :, 0].max(axis=1), kind="stable")]
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    xd = torch.from_numpy(x).cuda().to(tdt)
    ctx, pools, _ = _pools(n + 40, n_kv, d, dtype, n + 10 if slab else 10)
    if slab:
        sid, at = ctx.hot_alloc(n)
        ctx.hot_fill(0, sid, xd, xd)
        slots = np.arange(at, at + n)
    else:
        slots = (10 + rng.permutation(n + 30)[:n]).astype(np.int32)
        ctx.cold_append(0, xd, xd, torch.from_numpy(slots).cuda(), n)
    ctx.sync_status()
    for pool in pools:
        _same_bytes(pool.cpu().numpy()[slots], xd.float().cpu().numpy(), BLOCK if slab else 1, n_kv, d)


def test_token_write_refuses_bad_slots(cuda_ok):
    torch, gb, rng = _torch(), _gb(), np.random.default_rng(5)
    c = Kv4(rng, n_q=2, n_kv=2, d=64, dtype="bf16", prefixes=[10])
    before = c.kp.clone()
    x = c.to(_rows(rng, 3, 2, 64, "bf16"))
    c.ctx.cold_append(0, x, x, torch.tensor([0, -1, c.kp.shape[0]], dtype=torch.int32, device="cuda"), 3)
    with pytest.raises(gb.DeviceCheckFailed):
        c.ctx.sync_status()
    assert torch.equal(before, c.kp)


@pytest.mark.parametrize("n_kv,d,dtype", SHAPES)
@pytest.mark.parametrize("kind", ["kv4", "kv8", "plain"])
def test_read_gives_what_the_cache_holds(cuda_ok, n_kv, d, dtype, kind):
    """Slab ranges and scattered slots, one named twice; rows behind the last one are left as they were.
    4 bits and the plain cache: exact.  8 bits: the fp32 product of code and scale, rounded to the type (2^-24, then half a step)."""
    torch, rng = _torch(), np.random.default_rng([n_kv, d])
    L, N = 150, 77
    n_slots = L + N + 40
    ctx, pools, tdt = _pools(n_slots, n_kv, d, dtype, L + 5, kind)
    sid, _ = ctx.hot_alloc(L)
    pk, pv, ck, cv = (_odd_values(rng, _rows(rng, n, n_kv, d, dtype)) for n in (L, L, N, N))
    pk, pv, ck, cv = (torch.from_numpy(x).cuda().to(tdt) for x in (pk, pv, ck, cv))
    slots = torch.from_numpy((L + 5 + rng.permutation(N + 30)[:N]).astype(np.int32)).cuda()
    ctx.hot_fill(0, sid, pk, pv)
    ctx.cold_append(0, ck, cv, slots, N)

    def held(x, block):
        x = x.float().cpu().numpy()
        if kind == "plain":
            return x.astype(np.float64)
        return (K4 if kind == "kv4" else K8).through_cache(x, block)

    def check(got, want, n):
        tail = got[n:]
        assert torch.isnan(tail).all()
        got = got[:n].double().cpu().numpy()
        if kind != "kv8":
            assert np.array_equal(got, want, equal_nan=True)
        else:
            tol = (2.0 ** -24 + (2.0 ** -8 if dtype == "bf16" else 0.0)) * 1.01 * np.abs(want) + 2.0 ** -133
            assert ((np.abs(got - want) <= tol) | (np.isnan(got) & np.isnan(want))).all()

    order = rng.permutation(N)
    order[3] = order[9]
    for t0, n in ((0, L), (13, 1), (63, 66), (L - 1, 1), (L, 0)):
        k, v = (torch.full((n + 2, n_kv, d), float("nan"), dtype=tdt, device="cuda") for _ in range(2))
        ctx.hot_read(0, sid, t0, n, k, v)
        ctx.sync_status()
        check(k, held(pk, BLOCK)[t0:t0 + n], n)
        check(v, held(pv, BLOCK)[t0:t0 + n], n)
    for n in (N, 1, 33, 0):
        k, v = (torch.full((n + 2, n_kv, d), float("nan"), dtype=tdt, device="cuda") for _ in range(2))
        ctx.cold_read(0, slots[torch.from_numpy(order).cuda()].contiguous(), n, k, v)
        ctx.sync_status()
        check(k, held(ck, 1)[order[:n]], n)
        check(v, held(cv, 1)[order[:n]], n)


@pytest.mark.parametrize("kind", ["kv4", "kv8", "plain"])
def test_read_leaves_the_rows_of_bad_slots(cuda_ok, kind):
    torch, gb = _torch(), _gb()
    ctx, pools, tdt = _pools(60, 2, 64, "bf16", 10, kind)
    x = torch.randn(50, 2, 64, device="cuda").to(tdt)
    ctx.cold_append(0, x, x, torch.arange(10, 60, dtype=torch.int32, device="cuda"), 50)
    k, v = (torch.full((5, 2, 64), 7.0, dtype=tdt, device="cuda") for _ in range(2))
    ctx.cold_read(0, torch.tensor([12, 9, -1, 60, 59], dtype=torch.int32, device="cuda"), 5, k, v)
    with pytest.raises(gb.DeviceCheckFailed):
        ctx.sync_status()
    for y in (k, v):
        assert (y[1:4] == 7.0).all() and not (y[[0, 4]] == 7.0).all(dim=2).any()


@pytest.mark.parametrize("n_kv,d,dtype", [(8, 128, "bf16"), (2, 64, "f32"), (3, 96, "bf16"), (1, 32, "f32")])
@pytest.mark.parametrize("kind", ["kv4", "kv8", "plain"])
def test_rows_on_16_byte_boundaries_only(cuda_ok, n_kv, d, dtype, kind):
    """Rows and results that start 16 bytes past a 32-byte boundary: the same bytes and values as from one."""
    torch, rng = _torch(), np.random.default_rng([n_kv, d, 16])
    L, N = 130, 40

    def once(off):
        rng = np.random.default_rng(7)
        ctx, pools, tdt = _pools(L + N + 20, n_kv, d, dtype, L + 5, kind)
        sid, _ = ctx.hot_alloc(L)
        step = off // torch.tensor([], dtype=tdt).element_size()

        def place(n):
            x = torch.empty(n * n_kv * d + step, dtype=tdt, device="cuda")[step:].view(n, n_kv, d)
            assert x.data_ptr() % 32 == off
            return x
        pk, pv, ck, cv = (place(n) for n in (L, L, N, N))
        for x in (pk, pv, ck, cv):
            x.copy_(torch.from_numpy(_rows(rng, x.shape[0], n_kv, d, dtype)))
        slots = torch.from_numpy((L + 5 + rng.permutation(N + 15)[:N]).astype(np.int32)).cuda()
        ctx.hot_fill(0, sid, pk, pv)
        ctx.cold_append(0, ck, cv, slots, N)
        outs = [place(n) for n in (L, L, N, N)]
        ctx.hot_read(0, sid, 0, L, outs[0], outs[1])
        ctx.cold_read(0, slots, N, outs[2], outs[3])
        ctx.sync_status()
        return [p.clone() for p in pools] + outs

    for a, b in zip(once(0), once(16)):
        assert torch.equal(a.view(torch.uint8) if a.dtype != torch.uint8 else a, b.contiguous().view(torch.uint8) if b.dtype != torch.uint8 else b)


def test_rows_go_through_the_cache_unchanged_the_second_time(cuda_ok):
    """What a COLD token reads back as is held exactly when it is written again."""
    torch, rng = _torch(), np.random.default_rng(6)
    ctx, _, tdt = _pools(400, 8, 128, "bf16", 10)
    x = torch.from_numpy(_rows(rng, 150, 8, 128, "bf16")).cuda().to(tdt)
    k, v, k2, v2 = (torch.empty_like(x) for _ in range(4))
    for src, dst, at in (((x, x.flip(0).contiguous()), (k, v), 10), ((k, v), (k2, v2), 200)):
        slots = torch.arange(at, at + 150, dtype=torch.int32, device="cuda")
        ctx.cold_append(0, *src, slots, 150)
        ctx.cold_read(0, slots, 150, *dst)
    ctx.sync_status()
    want = K4.through_cache(K4.through_cache(x.float().cpu().numpy(), 1).astype(np.float32), 1)
    assert np.array_equal(k2.double().cpu().numpy(), want)


# ---- attention --------------------------------------------------------------------------------

HEADS = [(32, 8, 128, "bf16"), (40, 8, 128, "bf16"), (4, 4, 128, "bf16"), (7, 1, 128, "bf16"), (16, 2, 128, "bf16"), (6, 3, 128, "bf16"),
         (24, 2, 128, "bf16"), (8, 2, 64, "f32"), (9, 3, 96, "bf16"), (4, 2, 256, "f32"), (20, 1, 32, "f32"), (10, 10, 128, "bf16"),
         (32, 16, 128, "bf16"), (18, 9, 128, "bf16"), (8, 2, 64, "bf16"), (12, 1, 64, "bf16"), (24, 12, 64, "bf16"), (5, 5, 192, "bf16")]


@pytest.mark.parametrize("n_q,n_kv,d,dtype", HEADS)
def test_decode_matches_64_bit(cuda_ok, n_q, n_kv, d, dtype):
    """Ragged prefixes with a prefix-less, a prefix-only and a one-token request."""
    rng = np.random.default_rng([n_q, n_kv, d])
    c = Kv4(rng, n_q=n_q, n_kv=n_kv, d=d, dtype=dtype, prefixes=[517, 130], of=[0, 1, -1, 0, 0, 1, 0, -1, 0],
            lens=[5, 33, 70, 0, 1, 16, 200, 17, 64], slots_before=9)
    c.check(*c.decode(), f"{n_q}/{n_kv}/{d}/{dtype}")


@pytest.mark.parametrize("L_p", [1, 15, 63, 64, 65, 127, 128, 129, 300, 1000])
@pytest.mark.parametrize("d", [128, 64])
def test_decode_prefix_lengths(cuda_ok, L_p, d):
    rng = np.random.default_rng([L_p, d])
    c = Kv4(rng, n_q=32, n_kv=8, d=d, dtype="bf16", prefixes=[L_p], of=[0, 0], lens=[0, 3], slots_before=L_p % 7)
    c.check(*c.decode(), f"L_p {L_p}")


@pytest.mark.parametrize("n_q,n_kv,d,dtype", [(32, 8, 128, "bf16"), (16, 2, 64, "bf16"), (24, 2, 128, "bf16"), (8, 2, 64, "f32")])
def test_decode_requests_without_keys(cuda_ok, n_q, n_kv, d, dtype):
    """o = 0 and lse = -inf where a request has no prefix and, by the device's length, no token (by the host's it is
    refused); the others are not touched by it."""
    torch, gb = _torch(), _gb()
    rng = np.random.default_rng([n_q, d])
    lens = [40, 7, 0, 3]
    c = Kv4(rng, n_q=n_q, n_kv=n_kv, d=d, dtype=dtype, prefixes=[70], of=[-1, -1, 0, 0], lens=lens)
    slabs = [-1, -1, c.slabs[0], c.slabs[0]]
    with pytest.raises(gb.GranikvError):
        c.ctx.dispatch(gb.Batch(slabs, [40, 0, 0, 3], c.table, c.cap))
    c.live[1] = 0
    o, lse = c.decode(batch=gb.Batch(slabs, lens, c.table, c.cap, seq_len_dev=c.live))
    assert (o[1] == 0).all() and torch.isneginf(lse[1]).all()
    rows = [0, 2, 3]
    c.of, c.lens, c.q_host = [c.of[b] for b in rows], [lens[b] for b in rows], c.q_host[rows]
    c.ck, c.cv, c.cu = ([x[b] for b in rows] for x in (c.ck, c.cv, c.cu))
    c.check(o[rows], lse[rows], "the others")


@pytest.mark.parametrize("L_p", [1, 33, 64, 129])
@pytest.mark.parametrize("d", [128, 64])
def test_decode_slab_that_ends_the_pool(cuda_ok, L_p, d):
    """One slot behind the slab: tiles and boxes reach past the pool."""
    rng = np.random.default_rng([L_p, d, 1])
    c = Kv4(rng, n_q=8, n_kv=2, d=d, dtype="bf16", prefixes=[L_p], of=[0], lens=[1], holes=0)
    assert c.kp.shape[0] == L_p + 1
    c.check(*c.decode(), f"L_p {L_p}")


@pytest.mark.parametrize("L_p", [640, 777, 2048, 5000])
@pytest.mark.parametrize("d", [128, 64])
def test_decode_long_prefix_pieces(cuda_ok, L_p, d):
    """Few CTAs, so that a piece has many tiles: its rings and buffers come round again and again."""
    rng = np.random.default_rng([L_p, d])
    c = Kv4(rng, n_q=64, n_kv=8, d=d, dtype="bf16", prefixes=[L_p], of=[0] * 160, lens=[0] * 160)
    assert c.ctx.dispatch(c.batch).groups()[0]["n_splits"] <= 2
    o, lse = c.decode()
    rows = [0, 1, 15, 16, 17, 80, 158, 159]
    c.of, c.lens, c.q_host = [0] * len(rows), [0] * len(rows), c.q_host[rows]
    c.ck, c.cv, c.cu = c.ck[:len(rows)], c.cv[:len(rows)], c.cu[:len(rows)]
    c.check(o[rows], lse[rows], f"L_p {L_p}")


@pytest.mark.parametrize("B", [1, 3, 33, 100])
@pytest.mark.parametrize("n_q", [8, 40, 64])
@pytest.mark.parametrize("d", [128, 64])
def test_decode_rows_of_a_group(cuda_ok, B, n_q, d):
    """From one row a KV head to several row blocks, the group's requests scattered over the batch."""
    rng = np.random.default_rng([B, n_q, d])
    c = Kv4(rng, n_q=n_q, n_kv=8, d=d, dtype="bf16", prefixes=[390, 64], of=[b * 7 % 3 % 2 for b in range(B)],
            lens=[int(x) for x in rng.integers(0, 20, B)])
    c.check(*c.decode(), f"B {B} n_q {n_q}")


@pytest.mark.parametrize("lens", [[1], [15], [16], [17], [31, 1], [5000], [1, 2, 3, 4, 700, 5], [33] * 50])
@pytest.mark.parametrize("n_q,n_kv,d", [(32, 8, 128), (24, 12, 128), (3, 1, 128), (32, 8, 64), (36, 9, 64), (10, 5, 64)])
def test_decode_cold_lengths(cuda_ok, lens, n_q, n_kv, d):
    rng = np.random.default_rng(sum(lens))
    c = Kv4(rng, n_q=n_q, n_kv=n_kv, d=d, dtype="bf16", of=[-1] * len(lens), lens=lens)
    c.check(*c.decode(), f"COLD {lens[:4]}")


@pytest.mark.parametrize("d", [128, 64])
def test_decode_peaked_and_uneven_scales(cuda_ok, d):
    """Scores far apart, and blocks, tokens and groups of 16 whose K or V differ by many powers of two."""
    def edit(kind, k, v):
        n = k.shape[0]
        if kind == "prefix":
            v[:64] *= np.float32(2.0 ** -12)
            v[64:128] *= np.float32(2.0 ** 10)
            k[:64] *= np.float32(2.0 ** 3)
            k[128:192] *= np.float32(2.0 ** -20)
        for t in range(0, n, 3):
            v[t] *= np.float32(2.0 ** ((t % 31) - 15))
        for c in range(0, k.shape[2], 16):
            k[:, :, c:c + 16] *= np.float32(2.0 ** (-(c // 16) % 5))
            v[:, :, c:c + 16] *= np.float32(2.0 ** ((c // 16) * 3 % 7 - 3))
    rng = np.random.default_rng(11)
    c = Kv4(rng, n_q=32, n_kv=8, d=d, dtype="bf16", prefixes=[700], of=[0, 0, -1], lens=[100, 0, 300], q_scale=2.0, edit=edit)
    c.check(*c.decode(), "uneven")


def test_decode_zero_rows(cuda_ok):
    """All-zero K (equal scores) and all-zero V blocks."""
    def edit(kind, k, v):
        k[:] = 0.0
        v[: k.shape[0] // 2] = 0.0
    rng = np.random.default_rng(12)
    c = Kv4(rng, n_q=16, n_kv=4, d=128, dtype="bf16", prefixes=[200], of=[0, -1], lens=[20, 40], edit=edit)
    c.check(*c.decode(), "zeros")


def test_decode_large_queries(cuda_ok):
    """q beyond fp16's range in some rows (bf16 holds it), tiny in others."""
    rng = np.random.default_rng(13)
    c = Kv4(rng, n_q=8, n_kv=2, d=128, dtype="bf16", prefixes=[150], of=[0, 0, -1], lens=[10, 0, 30], edit=lambda kind, k, v: k.__imul__(np.float32(2.0 ** -17)))
    torch = _torch()
    scale = torch.tensor([2.0 ** 18, 2.0 ** 17, 1.0, 2.0 ** -30, 2.0 ** 16, 0.0, 2.0 ** -3, 2.0 ** 14], device="cuda")[None, :, None]
    c.q = (c.q.float() * scale).to(torch.bfloat16)
    c.q_host = c.q.float().cpu().numpy().astype(np.float64)
    c.check(*c.decode(), "large q")


@pytest.mark.parametrize("L_p", [1, 70, 200])
@pytest.mark.parametrize("size", [2.0 ** -30, 2.0 ** -40, 2.0 ** -100])
def test_decode_tiny_queries_over_zero_keys(cuda_ok, L_p, size):
    """All-zero K and a q so small that the product of the scales underflows: the weights are equal, the places
    past the prefix's end still have none."""
    def edit(kind, k, v):
        k[:] = 0.0
    c = Kv4(np.random.default_rng(33), n_q=32, n_kv=8, d=128, dtype="bf16", prefixes=[L_p], of=[0, 0, -1], lens=[0, 5, 9], q_scale=size, edit=edit)
    c.check(*c.decode(), f"{L_p} {size}")


@pytest.mark.parametrize("n_q,n_kv,d,dtype", [(16, 4, 128, "bf16"), (8, 2, 64, "f32"), (16, 4, 64, "bf16")])
@pytest.mark.parametrize("where", ["prefix", "cold"])
def test_decode_nan_value_stays_with_its_columns(cuda_ok, n_q, n_kv, d, dtype, where):
    """A NaN in one head of one token's V reaches its 16 columns of that head's output of the requests that
    attend it, and nothing else."""
    torch = _torch()

    def case(edit):
        return Kv4(np.random.default_rng(14), n_q=n_q, n_kv=n_kv, d=d, dtype=dtype, prefixes=[100], of=[0, -1, 0], lens=[20, 40, 5], edit=edit)

    def edit(kind, k, v):
        if kind == where and k.shape[0] in (100, 40):
            v[3, 1, 37] = np.nan

    (o, lse), (o2, lse2) = (case(e).decode() for e in (None, edit))
    hit = torch.zeros_like(o, dtype=torch.bool)
    g = n_q // n_kv
    for b in [0, 2] if where == "prefix" else [1]:
        hit[b, g:2 * g, 32:48] = True
    assert torch.equal(torch.isnan(o2), hit)
    assert not torch.isnan(lse2).any() and torch.equal(lse2, lse)
    # (the block's other elements may stand on another exponent or scale than without the NaN)
    rest = torch.ones_like(hit)
    for b in [0, 2] if where == "prefix" else [1]:
        rest[b, g:2 * g] = False
    assert torch.equal(o2[rest], o[rest])


@pytest.mark.parametrize("shape", [(32, 8, 128, "bf16"), (8, 2, 64, "f32"), (32, 8, 64, "bf16")])
@pytest.mark.parametrize("where", ["prefix", "cold"])
def test_decode_nan_key_reaches_its_readers(cuda_ok, shape, where):
    """A NaN in one head of one token's K makes that head NaN for the requests that attend the token."""
    torch = _torch()
    n_q, n_kv, d, dtype = shape

    def case(edit):
        return Kv4(np.random.default_rng(26), n_q=n_q, n_kv=n_kv, d=d, dtype=dtype, prefixes=[300], of=[0, -1, 0], lens=[20, 40, 0], edit=edit)

    def edit(kind, k, v):
        if kind == where and k.shape[0] in (300, 40):
            k[17, 1, 9] = np.nan

    (o, lse), (o2, lse2) = (case(e).decode() for e in (None, edit))
    g = n_q // n_kv
    hit = torch.zeros_like(lse, dtype=torch.bool)
    hit[[0, 2] if where == "prefix" else [1], g:2 * g] = True
    assert torch.equal(torch.isnan(lse2), hit) and torch.isnan(o2[hit]).all()
    assert torch.equal(o2[~hit], o[~hit]) and torch.equal(lse2[~hit], lse[~hit])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("backend", ["dense", "cascade"])
def test_decode_bad_query_stays_with_its_head(cuda_ok, bad, backend):
    """A NaN or infinity in one head's q makes that head's row NaN and changes no other."""
    torch, gb, rng = _torch(), _gb(), np.random.default_rng(23)
    c = Kv4(rng, n_q=32, n_kv=8, d=128, dtype="bf16", prefixes=[300], of=[0, 0, -1], lens=[20, 0, 70],
            backend=gb.BACKEND_DENSE if backend == "dense" else gb.BACKEND_CASCADE)
    o, lse = c.decode()
    for b, h in ((0, 5), (1, 31), (2, 0)):
        c.q[b, h, 77] = bad
    o2, lse2 = c.decode()
    hit = torch.zeros_like(lse, dtype=torch.bool)
    hit[0, 5] = hit[1, 31] = hit[2, 0] = True
    assert torch.equal(torch.isnan(o2).any(dim=2), hit) and torch.isnan(o2[hit]).all() and torch.equal(torch.isnan(lse2), hit)
    assert torch.equal(o2[~hit], o[~hit]) and torch.equal(lse2[~hit], lse[~hit])


@pytest.mark.parametrize("n_q,n_kv,d,dtype", [(32, 8, 128, "bf16"), (24, 2, 128, "bf16"), (9, 3, 96, "bf16"), (8, 2, 64, "f32"), (32, 8, 64, "bf16")])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf")])
def test_decode_infinite_query_over_keys_of_one_sign(cuda_ok, n_q, n_kv, d, dtype, bad):
    """Every K has the same sign in the dimension where q is infinite, so all scores of the head are -inf
    (or all +inf): its row is NaN all the same, with and without a slab, down to one token."""
    torch = _torch()

    def edit(kind, k, v):
        k[:, :, 7] = -np.abs(k[:, :, 7]) - 1.0

    c = Kv4(np.random.default_rng([n_q, d]), n_q=n_q, n_kv=n_kv, d=d, dtype=dtype, prefixes=[150], of=[0, -1, -1, 0], lens=[20, 1, 70, 0], edit=edit)
    o, lse = c.decode()
    hit = torch.zeros_like(lse, dtype=torch.bool)
    for b, h in ((0, 1), (1, 0), (2, n_q - 1), (3, 2)):
        c.q[b, h, 7] = bad
        hit[b, h] = True
    o2, lse2 = c.decode()
    assert torch.equal(torch.isnan(lse2), hit) and torch.isnan(o2[hit]).all()
    assert torch.equal(o2[~hit], o[~hit]) and torch.equal(lse2[~hit], lse[~hit])


def _uneven_v(e, small, where, of):
    """V of about 2^e, and of `small` 2^-e or nothing in some blocks of a slab or COLD tokens."""
    def edit(kind, k, v):
        if kind != of:
            return
        n, step = k.shape[0], BLOCK if kind == "prefix" else 1
        at = np.arange(n) // step
        low = {"first": at <= at[-1] // 2, "last": at > at[-1] // 2, "alternate": at % 2 == 1}[where] if n else np.zeros(0, bool)
        v[~low] *= np.float32(2.0 ** e)
        v[low] *= np.float32(small * 2.0 ** -e)
        k[low] *= np.float32(2.0)
    return edit


UNEVEN = [(32, 8, 128, "bf16"), (24, 2, 128, "bf16"), (8, 2, 64, "f32"), (32, 8, 64, "bf16")]


@pytest.mark.parametrize("n_q,n_kv,d,dtype", UNEVEN)
@pytest.mark.parametrize("e", [20, 62, 100])
@pytest.mark.parametrize("small", [0.0, 1.0])
@pytest.mark.parametrize("where", ["first", "last", "alternate"])
@pytest.mark.parametrize("of", ["cold", "prefix"])
def test_decode_values_far_apart(cuda_ok, n_q, n_kv, d, dtype, e, small, where, of):
    """A token keeps its weight in o and lse however small its V (or its block's) is beside the others'."""
    rng = np.random.default_rng([e, n_q])
    edit = _uneven_v(e, small, where, of)
    if of == "cold":
        c = Kv4(rng, n_q=n_q, n_kv=n_kv, d=d, dtype=dtype, prefixes=[90], of=[-1, -1, -1, 0], lens=[100, 2, 300, 40], edit=edit)
    else:
        c = Kv4(rng, n_q=n_q, n_kv=n_kv, d=d, dtype=dtype, prefixes=[1100, 300], of=[0, 1, 0, 1], lens=[0, 3, 20, 0], edit=edit)
    c.check(*c.decode(), f"{of} {e} {small} {where}")


def test_decode_long_cold_runs_of_zero_values(cuda_ok):
    """More than 600 COLD tokens of equal weight in one run, their V all zero: o is 0 and lse finite."""
    def edit(kind, k, v):
        if kind == "cold":
            k[:] = 0.0
            v[:] = 0.0
    c = Kv4(np.random.default_rng(31), n_q=4, n_kv=1, d=128, dtype="bf16", prefixes=[19200], of=[0, -1], lens=[1500, 1500], edit=edit)
    c.ctx.set_concurrency(True, 0.99)
    o, lse = c.decode()
    assert not o[1].any()
    c.check(o, lse, "zero V")


@pytest.mark.parametrize("n_q,n_kv,d,dtype", [(32, 8, 128, "bf16"), (8, 2, 64, "f32"), (6, 3, 128, "bf16"), (5, 5, 96, "bf16"), (24, 12, 128, "bf16"), (32, 8, 64, "bf16")])
@pytest.mark.parametrize("on_device", [False, True])
def test_fused_append_equals_append_then_decode(cuda_ok, n_q, n_kv, d, dtype, on_device):
    torch, gb, rng = _torch(), _gb(), np.random.default_rng(15)
    lens = [1, 16, 17, 40]
    c = Kv4(rng, n_q=n_q, n_kv=n_kv, d=d, dtype=dtype, prefixes=[70], of=[0, 0, -1, 0], lens=lens)
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
    for b in range(4):
        c.set_newest(b, k[b].float().cpu().numpy(), v[b].float().cpu().numpy())
    c.check(o1, lse1, "append")


def test_decode_in_a_graph_on_another_stream(cuda_ok):
    """Captured once and replayed with new q and growing live lengths; two graphs share one workspace and
    replay in turn."""
    torch, gb, rng = _torch(), _gb(), np.random.default_rng(16)
    lens = [30, 9, 64]
    c = Kv4(rng, n_q=32, n_kv=8, d=128, dtype="bf16", prefixes=[200], of=[0, -1, 0], lens=lens)
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
    full = [list(x) for x in (c.ck, c.cv, c.cu)]
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
        c.lens = live
        c.ck, c.cv, c.cu = ([x[:n] for x, n in zip(part, live)] for part in full)
        for og, lg in outs:
            c.check(og, lg, f"replay {live}")
    c.ctx.sync_status()


def test_step_of_calls_in_a_graph(cuda_ok):
    """Append, decode, read and weigh of a step captured together on a stream of their own and replayed with
    other rows: the results of the same calls made one by one."""
    torch, gb, rng = _torch(), _gb(), np.random.default_rng(40)
    lens = [30, 9, 64]
    c = Kv4(rng, n_q=32, n_kv=8, d=128, dtype="bf16", prefixes=[200], of=[0, -1, 0], lens=lens)
    batch = gb.Batch([c.slabs[i] if i >= 0 else -1 for i in c.of], lens, c.table, c.cap, c.live)
    plan = c.ctx.dispatch(batch)
    ws = torch.empty(c.ctx.workspace_size(plan), dtype=torch.uint8, device="cuda")
    newest = torch.stack([c.table[b, n - 1] for b, n in enumerate(lens)])
    k, v = (c.to(_rows(rng, 3, 8, 128, "bf16")) for _ in range(2))

    def buffers():
        return [torch.zeros_like(c.q), torch.zeros(c.q.shape[:2], device="cuda"), torch.zeros_like(k), torch.zeros_like(v),
                torch.zeros(3, c.cap, device="cuda")]

    def step(out, s):
        c.ctx.decode_attention_append(0, c.q, k, v, batch, plan, out[0], out[1], ws, ws.numel(), s)
        c.ctx.cold_read(0, newest, 3, out[2], out[3], s)
        c.ctx.cold_weigh(0, c.q, out[1], batch, out[4], 0.0, s)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    eager, replayed = buffers(), buffers()
    step(eager, s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step(replayed, s)
    for _ in range(3):
        k.copy_(c.to(_rows(rng, 3, 8, 128, "bf16")))
        v.copy_(c.to(_rows(rng, 3, 8, 128, "bf16")))
        c.q.copy_(torch.randn_like(c.q))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        s.synchronize()
        got = [x.clone() for x in replayed]
        step(eager, s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager))
        for b in range(3):
            c.set_newest(b, k[b].float().cpu().numpy(), v[b].float().cpu().numpy())
        c.q_host = c.q.double().cpu().numpy()
        c.check(got[0], got[1], "step")
        assert np.array_equal(got[2].double().cpu().numpy(), K4.through_cache(k.float().cpu().numpy(), 1))
    c.ctx.sync_status()


@pytest.mark.parametrize("B,d", [(1, 128), (8, 128), (64, 128), (8, 64)])
def test_calls_back_to_back_in_a_graph(cuda_ok, B, d):
    """Two dozen calls one after the other, replayed again and again (as many prefix CTAs as SMs, and fewer): every one
    ends, with the result of a single call."""
    torch, rng = _torch(), np.random.default_rng([B, 41])
    c = Kv4(rng, n_q=32, n_kv=8, d=d, dtype="bf16", prefixes=[9728], of=[0] * B, lens=[0] * B)
    o, lse = c.decode()
    plan = c.ctx.dispatch(c.batch)
    ws = torch.empty(c.ctx.workspace_size(plan), dtype=torch.uint8, device="cuda")
    outs = [(torch.zeros_like(o), torch.zeros_like(lse)) for _ in range(24)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.ctx.decode_attention(0, c.q, c.batch, plan, *outs[0], ws, ws.numel(), s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        for a, b in outs:
            c.ctx.decode_attention(0, c.q, c.batch, plan, a, b, ws, ws.numel(), s)
    for _ in range(20):
        with torch.cuda.stream(s):
            g.replay()
    s.synchronize()
    c.ctx.sync_status()
    for a, b in outs:
        assert torch.equal(a, o) and torch.equal(b, lse)


def test_decode_far_slots(cuda_ok):
    """Slots whose byte offsets pass 2^32, in slab and COLD pool."""
    torch, gb, rng = _torch(), _gb(), np.random.default_rng(17)
    n_kv, d, n_q = 8, 128, 32
    row = gb.kv4_row_bytes(n_kv, d)
    n_slots = 2 ** 33 // row + 4000
    kp, vp = (torch.zeros((n_slots, row), dtype=torch.uint8, device="cuda") for _ in range(2))
    n_hot = n_slots - 2000
    ctx = gb.Context(n_layers=1, n_q=n_q, n_kv=n_kv, head_dim=d, dtype=gb.DTYPE_BF16, n_slots=n_slots, k_pools=[kp], v_pools=[vp],
                     hot_fraction=(n_hot + 0.5) / n_slots, kv4=True, max_batch=4)
    ctx.hot_alloc(n_hot - 300)
    sid, off = ctx.hot_alloc(300)
    assert off * row > 2 ** 32
    c = Kv4(rng, n_q=n_q, n_kv=n_kv, d=d, dtype="bf16", prefixes=[300], of=[0, -1], lens=[40, 60])
    table = torch.full((2, 64), -1, dtype=torch.int32, device="cuda")
    table[0, :40] = torch.arange(n_slots - 40, n_slots, device="cuda")
    table[1, :60] = torch.arange(n_slots - 200, n_slots - 140, device="cuda").flip(0)
    pk, pv = c.pk[0].astype(np.float32), c.pv[0].astype(np.float32)
    ctx.hot_fill(0, sid, c.to(pk), c.to(pv))
    for b, n in enumerate([40, 60]):
        k, v = c.ck[b].astype(np.float32), c.cv[b].astype(np.float32)
        ctx.cold_append(0, c.to(k), c.to(v), table[b, :n].contiguous(), n)
        c.ck[b], c.cv[b], c.cu[b] = K4.through_cache(k, 1), K4.through_cache(v, 1), K4.units(v, 1)
    c.pk, c.pv, c.pu = [K4.through_cache(pk, BLOCK)], [K4.through_cache(pv, BLOCK)], [K4.units(pv, BLOCK)]
    k, v = (torch.empty(300, n_kv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ctx.hot_read(0, sid, 0, 300, k, v)
    assert np.array_equal(k.double().cpu().numpy(), c.pk[0]) and np.array_equal(v.double().cpu().numpy(), c.pv[0])
    ctx.cold_read(0, table[0, :40].contiguous(), 40, k, v)
    assert np.array_equal(k[:40].double().cpu().numpy(), c.ck[0])
    c.ctx, c.batch = ctx, gb.Batch([sid, -1], [40, 60], table, 64)
    c.check(*c.decode(), "far slots")


def test_decode_bad_slot_is_latched(cuda_ok):
    gb, rng = _gb(), np.random.default_rng(18)
    c = Kv4(rng, n_q=32, n_kv=8, d=128, dtype="bf16", of=[-1, -1], lens=[40, 20])
    c.table[0, 7] = c.kp.shape[0] + 5
    with pytest.raises(gb.DeviceCheckFailed):
        c.decode()
    c.table[0, 7] = -3
    with pytest.raises(gb.DeviceCheckFailed):
        c.decode()


def test_stalled_wait_is_reported_and_the_context_survives(cuda_ok):
    gb, rng = _gb(), np.random.default_rng(30)
    c = Kv4(rng, n_q=32, n_kv=8, d=128, dtype="bf16", prefixes=[300], of=[0, 0, -1], lens=[40, 20, 70])
    c.check(*c.decode(), "before")
    c.ctx.inject_stall(True)
    with pytest.raises(gb.DeviceCheckFailed):
        c.decode()
    c.check(*c.decode(), "after")


def test_prefill_is_refused_and_static_workspace_serves(cuda_ok):
    torch, gb, rng = _torch(), _gb(), np.random.default_rng(19)
    c = Kv4(rng, n_q=32, n_kv=8, d=128, dtype="bf16", prefixes=[100], of=[0], lens=[20])
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


SCHEDULES = {"serial": lambda x: x.set_concurrency(False), "half": lambda x: x.set_concurrency(True, 0.5),
             "all": lambda x: x.set_concurrency(True, 1.0), "ahead": lambda x: x.set_dense_l2_ahead(4),
             "unfused": lambda x: x.set_fused_merge(False), "fused": lambda x: x.set_fused_merge(True),
             "mixed": lambda x: x.set_msat(30), "cascade": lambda x: x.set_msat(10000)}


@pytest.mark.parametrize("how", sorted(SCHEDULES))
@pytest.mark.parametrize("d", [128, 64])
def test_decode_schedules(cuda_ok, how, d):
    """Every knob of the schedule leaves the result within the same tolerance; `mixed` runs one group
    on the tensor cores and one on CUDA cores."""
    rng = np.random.default_rng(22)
    c = Kv4(rng, n_q=32, n_kv=8, d=d, dtype="bf16", prefixes=[1500, 700], of=[0, 1, 0, 0, -1, 0, 0, 0, 0, 0], lens=[300, 20, 0, 1, 90, 64, 700, 33, 5, 16])
    SCHEDULES[how](c.ctx)
    c.check(*c.decode(), how)


def test_decode_on_two_streams_at_once(cuda_ok):
    """One plan, two workspaces, two streams: the results of the calls one after the other."""
    torch, rng = _torch(), np.random.default_rng(24)
    c = Kv4(rng, n_q=32, n_kv=8, d=128, dtype="bf16", prefixes=[2000], of=[0] * 8 + [-1], lens=[int(x) for x in rng.integers(0, 400, 8)] + [40])
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
    c = Kv4(rng, n_q=32, n_kv=8, d=128, dtype="bf16", prefixes=[90], of=[0, -1, 0], lens=[40, 35, 7])
    c.table[0, 3], c.table[0, 39], c.table[2, 6] = c.table[0, 4], c.table[0, 4], c.table[1, 20]
    for x in (c.ck, c.cv, c.cu):
        x[0][3] = x[0][39] = x[0][4]
        x[2][6] = x[1][20]
    c.check(*c.decode(), "twice")


# ---- weighing and eviction ---------------------------------------------------------------------

WEIGH = [(32, 8, 128, "bf16"), (40, 8, 128, "bf16"), (7, 1, 128, "bf16"), (64, 4, 128, "bf16"), (8, 2, 64, "f32"), (12, 12, 128, "bf16"),
         (9, 3, 96, "bf16"), (4, 2, 256, "f32"), (64, 64, 32, "f32"), (8, 2, 64, "bf16"), (33, 3, 64, "bf16"), (65, 65, 64, "bf16")]


@pytest.mark.parametrize("n_q,n_kv,d,dtype", WEIGH)
@pytest.mark.parametrize("keep", [0.0, 0.5])
def test_weigh_matches_64_bit(cuda_ok, n_q, n_kv, d, dtype, keep):
    """w = sum_h exp(s_h - lse_h).  A score errs by x (above) plus the rounding of s - lse, 2^-23 (|s| + |lse|), in the
    exponent; the exponential adds 2^-20 and the sum n_q 2^-24, each relative to w; keep * old adds 2^-23 of it."""
    torch, gb, rng = _torch(), _gb(), np.random.default_rng([n_q, n_kv, d])
    lens = [1, 0, 33, 150, 16, 17, 600]
    c = Kv4(rng, n_q=n_q, n_kv=n_kv, d=d, dtype=dtype, of=[-1] * len(lens), lens=lens)
    B = len(lens)
    batch = gb.Batch([-1] * B, lens, c.table, c.cap, c.live)
    s = [np.einsum("jgd,ljd->jgl", c.q_host[b].reshape(n_kv, -1, d), c.ck[b]).reshape(n_q, -1) / math.sqrt(d) for b in range(B)]
    lse = np.stack([np.log(np.exp(x).sum(axis=1) + rng.uniform(0, 5)) if x.shape[1] else np.zeros(n_q) for x in s])
    lse[2, 0] = -np.inf
    lse = torch.from_numpy(lse.astype(np.float32)).cuda()
    weight = torch.rand(B, c.cap, device="cuda")
    before = weight.double().cpu().numpy()
    c.ctx.cold_weigh(0, c.q, lse, batch, weight, keep)
    c.ctx.sync_status()
    again = torch.from_numpy(before.astype(np.float32)).cuda()
    c.ctx.cold_weigh(0, c.q, lse, batch, again, keep)
    assert torch.equal(weight, again)
    got, lse = weight.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, n in enumerate(lens):
        gone = np.isneginf(lse[b])[:, None]
        p = np.where(gone, 0.0, np.exp(s[b] - lse[b][:, None]))
        x = d * 2.0 ** -24 * np.einsum("jgd,ljd->jgl", np.abs(c.q_host[b]).reshape(n_kv, -1, d), np.abs(c.ck[b])).reshape(n_q, -1) / math.sqrt(d)
        x = x + 2.0 ** -39 * np.abs(c.q_host[b]).max() * np.abs(c.ck[b]).sum(axis=2).max(initial=0.0) / math.sqrt(d)
        rel = x + 2.0 ** -23 * (np.abs(s[b]) + np.where(gone, 0.0, np.abs(lse[b][:, None]))) + 2.0 ** -20
        old = keep * before[b, :n]
        tol = (p * rel).sum(axis=0) + n_q * 2.0 ** -24 * p.sum(axis=0) + 2.0 ** -23 * (np.abs(old) + p.sum(axis=0))
        err = np.abs(got[b, :n] - (p.sum(axis=0) + old))
        assert (err <= tol).all(), f"row {b}: off by {np.max(err / tol)} of the tolerance"
        assert np.array_equal(got[b, n:], before[b, n:])


def test_weigh_bad_slot_is_latched(cuda_ok):
    torch, gb, rng = _torch(), _gb(), np.random.default_rng(41)
    c = Kv4(rng, n_q=32, n_kv=8, d=128, dtype="bf16", of=[-1], lens=[40])
    c.table[0, 7] = c.kp.shape[0] + 5
    batch = gb.Batch([-1], [40], c.table, c.cap, c.live)
    weight = torch.ones(1, c.cap, device="cuda")
    c.ctx.cold_weigh(0, c.q, torch.zeros(1, 32, device="cuda"), batch, weight, 0.5)
    with pytest.raises(gb.DeviceCheckFailed):
        c.ctx.sync_status()
    assert weight[0, 7].item() == 0.5


# ---- the cache and the driver -------------------------------------------------------------------

def test_cache_in_4_bits_with_prefix_lifecycle(cuda_ok):
    """GraniKVCache(kv4=True): admission to HOT, fallback to COLD shared by two requests, appends, decode with
    the newest token written by the call, eviction, and what a row holds read back."""
    torch, gb = _torch(), _gb()
    from shared_prefix_kv_decode_gb300 import GraniKVCache
    rng = np.random.default_rng(21)
    cache = GraniKVCache(n_layers=1, n_q=32, n_kv=8, head_dim=128, dtype=gb.DTYPE_BF16, n_slots=2000, max_batch=4, cap=400, kv4=True)
    assert cache.k_pools[0].dtype == torch.uint8
    c = Kv4(rng, n_q=32, n_kv=8, d=128, dtype="bf16")  # draws and checks
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
    at = np.cumsum([0] + own)

    def rows_of(new, prefix, through):
        t = through(new, 1)
        p = [through(prefix[0], BLOCK), through(prefix[1], 1)]
        return [np.concatenate([p[min(b, 1)], t[at[b]:at[b + 1]], t[len(t) - 3 + b][None]]) for b in range(3)]

    c.of, c.lens = [-1] * 3, [1] * 3
    c.ck, c.cv, c.cu = rows_of(kn, ks, K4.through_cache), rows_of(vn, vs, K4.through_cache), rows_of(vn, vs, K4.units)
    c.q_host = q.double().cpu().numpy()
    c.check(o, lse, "cache")
    for b in range(3):
        k, v = cache.read(0, b)
        assert np.array_equal(k.double().cpu().numpy(), c.ck[b]) and np.array_equal(v.double().cpu().numpy(), c.cv[b])
    # a 16-bit cache takes what row 1 holds
    wide = GraniKVCache(n_layers=1, n_q=32, n_kv=8, head_dim=128, dtype=gb.DTYPE_BF16, n_slots=800, max_batch=1, cap=400)
    k, v = cache.read(0, 1)
    wide.append([k.shape[0]], [k], [v])
    o2, lse2 = wide.decode(0, q[1:2].contiguous(), wide.batch([-1], wide.seq_len_host[:1]))
    wide.ctx.sync_status(wide.stream())
    k2, v2 = wide.read(0, 0)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    # both are within the tolerance above and half a bf16 step (the 16-bit path rounds its weights to bf16: 2^-9 a weight)
    V = np.abs(c.cv[1]).max()
    assert (o2[0].double() - o[1].double()).abs().max().item() <= (2.0 ** -7 + 2.0 ** -8) * V
    # the lightest tokens leave
    cache.weigh(0, q, lse, batch)
    out = cache.evict([2, 4, 0], keep_last=1)
    cache.ctx.sync_status(cache.stream())
    assert out.numel() == 6 and cache.seq_len_host[:3] == [4, 264, 251]
    k, v = cache.read(0, 0)
    assert k.shape[0] == 304 and np.array_equal(k[:300].double().cpu().numpy(), c.ck[0][:300])


@pytest.mark.parametrize("graph", [False, True])
def test_driver_over_the_4_bit_cache(cuda_ok, graph):
    """Arrivals, completions and a COLD budget: the last step's attention of every request, from the host's copies of its
    logical K/V put through the format."""
    from shared_prefix_kv_decode_gb300.decode_driver import DecodeDriver
    drv = DecodeDriver(prefix_lens=[300, 170], n_layers=2, max_batch=8, cap=256, n_slots=4000, seed=3, graph=graph, kv4=True,
                       cold_budget=40, keep_last=8, keep_logical=True)
    for p, n in [(0, 20), (1, 45), (0, 33)]:
        drv.arrive(p, n)
    for i in range(9):
        if i == 4:
            drv.complete(1)
            drv.arrive(1, 12)
        drv.step()
    drv.ctx.sync_status(drv.cache.stream())
    assert any(t["evicted"] for t in drv.finish_trace())
    c = Kv4(np.random.default_rng(0), n_q=32, n_kv=8, d=128, dtype="bf16")
    c.of, c.lens = [r["prefix"] for r in drv.rows], [r["len"] for r in drv.rows]
    c.pk, c.pv, c.pu = ([f(kv[i][1], BLOCK) for kv in drv.prefix_kv] for f, i in ((K4.through_cache, 0), (K4.through_cache, 1), (K4.units, 1)))
    k, v = ([np.concatenate(r[x][1]) for r in drv.rows] for x in ("k", "v"))
    c.ck, c.cv, c.cu = [K4.through_cache(x, 1) for x in k], [K4.through_cache(x, 1) for x in v], [K4.units(x, 1) for x in v]
    c.q_host = drv.last_q[1].astype(np.float64)
    o, lse = drv.last_out
    c.check(o[:drv.B], lse[:drv.B], f"driver graph={graph}")
    for b in range(drv.B):
        slots = drv.cache.req_to_slot[b, :c.lens[b]].contiguous()
        kd, vd = (_torch().empty(c.lens[b], 8, 128, dtype=_torch().bfloat16, device="cuda") for _ in range(2))
        drv.ctx.cold_read(1, slots, c.lens[b], kd, vd)
        assert np.array_equal(kd.double().cpu().numpy(), c.ck[b]) and np.array_equal(vd.double().cpu().numpy(), c.cv[b])
