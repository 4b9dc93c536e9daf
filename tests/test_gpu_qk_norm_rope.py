"""Head norms, rotation and cache write in one pass against fp64 and, for what
is a bit copy, bit for bit.  Bounds: see step_reference."""

import numpy as np
import pytest
import torch

import oracle
import workloads
from tests import step_reference as ref
from tests.parity import bf16_bits, to_dev_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_50_gb300 import build
    build.build()
    import paged_kv_cache_50_gb300 as pa
    pa.lib()
    assert pa.pa_get_device_error() == 0
    return pa


def f64(t):
    return t.detach().double().cpu().numpy()


class Case:
    """Queries, keys and values as views of one packed projection whose rows
    are `pad` elements longer than they need; slots scattered, some -1."""

    def __init__(self, seed, T, hq, hkv, d, bs, fp8, pad=0, max_pos=5000, skip=0.1):
        g = torch.Generator("cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.T, self.hq, self.hkv, self.d, self.bs, self.fp8 = T, hq, hkv, d, bs, fp8
        w = (hq + 2 * hkv) * d + pad
        self.packed = torch.randn((T, w), generator=g, device="cuda").bfloat16()
        self.packed *= torch.exp(torch.randn((T, 1), generator=g, device="cuda")).bfloat16()
        self.q = self.packed[:, :hq * d].view(T, hq, d)
        self.k = self.packed[:, hq * d:(hq + hkv) * d].view(T, hkv, d)
        self.v = self.packed[:, (hq + hkv) * d:(hq + 2 * hkv) * d].view(T, hkv, d)
        self.qw = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).bfloat16()
        self.kw = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).bfloat16()
        self.nb = -(-T // bs) + 2
        slots = rng.permutation(self.nb * bs)[:T].astype(np.int64)
        slots[rng.random(T) < skip] = -1
        self.slots = slots
        self.pos = rng.integers(0, max_pos, T).astype(np.int32)
        shape = (self.nb, 2, bs, hkv, d)
        self.pool = (torch.randint(0, 0x78, shape, generator=g, device="cuda", dtype=torch.uint8)
                     if fp8 else torch.randn(shape, generator=g, device="cuda").bfloat16())
        self.max_pos = max_pos
        self.ks, self.vs = 0.031, 0.027

    def call(self, pa, norm=True, rot=None, interleaved=False, eps=1e-5, slots=None, pos=None,
             q=None, **kw):
        rot = self.d if rot is None else rot
        self.table = pa.rope_table(self.max_pos, rot, 10000.0) if rot else None
        f = pa.pa_qk_norm_rope_cache_fp8 if self.fp8 else pa.pa_qk_norm_rope_cache
        scales = (self.ks, self.vs) if self.fp8 else ()
        return f(self.q if q is None else q, self.k, self.v, self.pool,
                 torch.from_numpy(self.slots if slots is None else slots).cuda(), *scales,
                 q_weight=self.qw if norm else None, k_weight=self.kw if norm else None, eps=eps,
                 cos_sin=self.table,
                 positions=torch.from_numpy(self.pos if pos is None else pos).cuda() if rot else None,
                 interleaved=interleaved, **kw)

    def check(self, got, before, norm, interleaved, eps, what):
        table = None if self.table is None else self.table.cpu().numpy()
        rot = table is not None
        q, qm = ref.norm_rope(f64(self.q), f64(self.qw) if norm else None, eps, table,
                              self.pos if rot else None, interleaved)
        k, km = ref.norm_rope(f64(self.k), f64(self.kw) if norm else None, eps, table,
                              self.pos if rot else None, interleaved)
        slop = 2.0 ** -19
        err = np.abs(f64(got) - q) - (2.0 ** -8 * np.abs(q) + slop * qm)
        assert err.max(initial=0) <= 0, f"{what}: q beyond its bound by {err.max():.3e}"
        live = self.slots >= 0
        blk, off = self.slots[live] // self.bs, self.slots[live] % self.bs
        pool = self.pool.cpu()
        if self.fp8:
            codes = pool.numpy()
            kk = torch.from_numpy(codes[blk, 0, off]).view(torch.float8_e4m3fn).double().numpy()
            want = np.clip(k[live] / self.ks, -448, 448)
            tol = 2.0 ** -4 * np.abs(want) + 2.0 ** -10 + slop * km[live] / self.ks
            err = np.abs(kk - want) - tol
            assert err.max(initial=0) <= 0, f"{what}: k codes beyond their bound"
            vals = oracle.reshape_and_cache_fp8(
                bf16_bits(self.k.contiguous()), bf16_bits(self.v.contiguous()),
                before.numpy(), self.slots, self.bs, self.ks, self.vs)
            assert np.array_equal(codes[blk, 1, off], vals[blk, 1, off]), f"{what}: v codes"
        else:
            kk = f64(self.pool)[blk, 0, off]
            err = np.abs(kk - k[live]) - (2.0 ** -8 * np.abs(k[live]) + slop * km[live])
            assert err.max(initial=0) <= 0, f"{what}: k beyond its bound"
            assert np.array_equal(bf16_bits(self.pool)[blk, 1, off],
                                  bf16_bits(self.v.contiguous())[live]), f"{what}: v"
        rest = np.ones((self.nb, self.bs), bool)
        rest[blk, off] = False
        a = pool.view(torch.uint8).numpy().reshape(self.nb, 2, self.bs, -1)
        b = before.view(torch.uint8).numpy().reshape(self.nb, 2, self.bs, -1)
        keep = np.broadcast_to(rest[:, None], (self.nb, 2, self.bs))
        assert np.array_equal(a[keep], b[keep]), f"{what}: other slots changed"


HEADS = [(4, 2, 64, 16), (32, 8, 128, 16), (1, 1, 128, 48), (10, 2, 64, 32), (16, 16, 64, 256),
         (64, 8, 128, 64), (7, 7, 128, 16), (48, 1, 64, 16)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_norm_rope_cache(pa, heads, fp8):
    hq, hkv, d, bs = heads
    for n, (T, rot, inter, norm) in enumerate([(1, d, False, True), (5, d, True, True),
                                               (67, d // 2, False, True), (33, 16, True, True),
                                               (18, d, False, False), (9, 0, False, True),
                                               (301, d // 4, False, True), (40, d // 2, True, False)]):
        c = Case(100 * n + hq, T, hq, hkv, d, bs, fp8, pad=8 * (n % 3))
        before = c.pool.cpu().clone()
        got = c.call(pa, norm, rot, inter)
        assert pa.pa_get_device_error() == 0
        c.check(got, before, norm, inter, 1e-5, f"{heads} T={T} rot={rot} inter={inter} norm={norm}")


def test_many_tokens(pa):
    c = Case(3, 4099, 8, 2, 128, 16, False)
    before = c.pool.cpu().clone()
    c.check(c.call(pa), before, True, False, 1e-5, "4099 tokens")
    assert pa.pa_get_device_error() == 0


def test_far_positions_keep_their_angle(pa):
    c = Case(4, 64, 4, 2, 128, 16, False, max_pos=1 << 20)
    c.pos = (np.arange(64) + (1 << 20) - 64).astype(np.int32)
    before = c.pool.cpu().clone()
    got = c.call(pa)
    c.check(got, before, True, False, 1e-5, "far positions")
    k = np.arange(64)
    ang = c.pos[:, None].astype(np.float64) * 10000.0 ** (-k / 64)
    assert np.abs(c.table.cpu().numpy()[c.pos, :64] - np.cos(ang)).max() <= 2.0 ** -24


def test_in_place_and_streams(pa):
    """q_out = q where q is dense; the call on a stream of its own."""
    c = Case(5, 129, 32, 8, 128, 16, False)
    want = c.call(pa).clone()
    dense = c.q.contiguous()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.call(pa, q=dense, q_out=dense, stream=s)
    s.synchronize()
    assert got.data_ptr() == dense.data_ptr() and torch.equal(got, want)
    with pytest.raises(ValueError):
        c.call(pa, q_out=c.q)   # not dense
    assert torch.equal(c.call(pa, stream=s.cuda_stream), want)
    s.synchronize()


def test_zero_rows_and_large_values(pa):
    """A head of zeros stays zero; values whose squares need the whole fp32 range."""
    c = Case(6, 20, 4, 2, 64, 16, False, skip=0.0)
    c.packed[3] = 0
    c.packed[4] *= 2.0 ** 50
    c.packed[5] *= 2.0 ** -40
    before = c.pool.cpu().clone()
    got = c.call(pa, eps=1e-5)
    assert (got[3] == 0).all()
    c.check(got, before, True, False, 1e-5, "range")


def test_bad_slots_and_positions(pa):
    c = Case(7, 12, 4, 2, 64, 16, False, skip=0.0)
    before = c.pool.clone()
    slots, pos = c.slots.copy(), c.pos.copy()
    slots[2] = c.nb * c.bs
    slots[4] = -(1 << 40)
    pos[6], pos[7] = c.max_pos, -1
    want = c.call(pa).clone()
    full = c.pool.clone()
    c.pool.copy_(before)
    out = torch.full_like(want, 7.0)
    c.call(pa, slots=slots, pos=pos, q_out=out)
    assert pa.pa_get_device_error() == pa.PA_DEVERR_SLOT | pa.PA_DEVERR_POSITION
    ok = [t for t in range(12) if t not in (6, 7)]
    assert torch.equal(out[ok], want[ok]) and (out[[6, 7]] == 7.0).all()
    for t in range(12):
        b, o = divmod(int(c.slots[t]), c.bs)
        src = before if t in (2, 4, 6, 7) else full
        assert torch.equal(c.pool[b, :, o], src[b, :, o]), t


def test_equals_the_plain_cache_write(pa):
    """Without norm and rotation it is pa_reshape_and_cache and a copy."""
    b = workloads.tiny_paged()
    q, k, v = to_dev_bf16(b.q), to_dev_bf16(b.key), to_dev_bf16(b.value)
    p1, p2 = to_dev_bf16(b.pool), to_dev_bf16(b.pool)
    slots = torch.from_numpy(b.slot_mapping).cuda()
    pa.pa_reshape_and_cache(k, v, p1, slots)
    got = pa.pa_qk_norm_rope_cache(q, k, v, p2, slots)
    assert torch.equal(got, q) and torch.equal(p1.view(torch.int16), p2.view(torch.int16))


def test_fp8_codes_are_those_of_the_division(pa):
    """Every bf16 pattern (infinities, NaN, zeros of both signs among them) at
    scales that are powers of two, far out, or anything: the same codes as
    pa_reshape_and_cache_fp8, which divides."""
    v = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    v = v.view(512, 2, 64)
    q = torch.zeros((512, 2, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(512, device="cuda")
    rng = np.random.default_rng(12)
    scales = [2.0 ** e for e in (-126, -101, -100, -99, -20, -3, 0, 1, 7, 40, 99, 100, 101, 127)]
    scales += list(np.exp2(rng.uniform(-12, 12, 150))) + list(np.exp2(rng.uniform(-126, 127, 60)))
    scales += [1.5, 3.0, 1 / 3, 0.1, 1 + 2.0 ** -23, 2 - 2.0 ** -23, 448.0, 1 / 448, 1e-45, 3e38]
    for s in scales:
        s = float(np.float32(s))
        a, b = (torch.zeros((32, 2, 16, 2, 64), dtype=torch.uint8, device="cuda") for _ in range(2))
        pa.pa_qk_norm_rope_cache_fp8(q, v, v, a, slots, s, s)
        pa.pa_reshape_and_cache_fp8(v, v, b, slots, s, s)
        assert torch.equal(a, b), s


def test_argument_checks(pa):
    c = Case(8, 6, 4, 2, 64, 16, False)
    slots = torch.from_numpy(c.slots).cuda()
    pos = torch.from_numpy(c.pos).cuda()
    table = pa.rope_table(100, 64)
    ok = dict(q=c.q, key=c.k, value=c.v, kv_cache=c.pool, slot_mapping=slots, q_weight=c.qw,
              k_weight=c.kw, cos_sin=table, positions=pos)
    for bad in (dict(q=c.q.float()), dict(q=c.q[:, :, ::2]), dict(q=c.q.transpose(1, 2)),
                dict(key=c.k[:5]), dict(value=c.v.cpu()), dict(slot_mapping=slots.int()),
                dict(k_weight=None), dict(q_weight=c.qw[:32]), dict(positions=None),
                dict(positions=pos.long()), dict(cos_sin=table.double()),
                dict(q_out=torch.empty(6, 4, 32, dtype=torch.bfloat16, device="cuda")),
                dict(kv_cache=c.pool.view(torch.int16)), dict(kv_cache=c.pool[:, :1])):
        with pytest.raises((ValueError, TypeError, pa.PaError)):
            pa.pa_qk_norm_rope_cache(**{**ok, **bad})
    odd = torch.empty(6 * (8 * 64) + 4, dtype=torch.bfloat16, device="cuda")[4:].view(6, 8, 64)
    with pytest.raises(pa.PaError):   # not 16-byte aligned
        pa.pa_qk_norm_rope_cache(**{**ok, "q": odd[:, :4]})
