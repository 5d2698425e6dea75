"""dsa_cache_append against the float64 oracle.

Tolerances: the latent's normalised dims 2^-18 relative before their rounding to bf16 (16 fused adds in a
chain, 5 tree steps: 2^-19; see the norm's tests), rotated values 2^-20 of (|a| + |b|) (see the rotation's);
the key's scale is the largest of those over 448; codes half an e4m3 step."""
import numpy as np
import pytest
import torch

import oracle
import sparse_attention_09_b200 as dsa

pytestmark = pytest.mark.gpu
EPS = 1e-6
ROPE = {False: dsa.DSA_ROPE_INTERLEAVED, True: dsa.DSA_ROPE_HALF}


def rnd(shape, seed):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def f64(t):
    return t.double().cpu().numpy()


class Caches:
    """Paged caches of B sequences with scattered pages, filled with a pattern that no append writes."""

    def __init__(self, B, pages, d_I, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.table = torch.randperm(B * pages + 2, generator=g)[:B * pages].reshape(B, pages).int().cuda()
        n = B * pages + 2
        self.latent = torch.full((n, 64, 576), 7.0, dtype=torch.bfloat16, device="cuda")
        self.codes = torch.full((n, 64, d_I), 0x55, dtype=torch.uint8, device="cuda")
        self.scale = torch.full((n, 64), 5.0, device="cuda")
        self.ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.describe(pages * 64)

    def describe(self, max_len):
        self.lat_desc = dsa.paged_desc(self.latent, self.table, self.ctx, max_len)
        self.key_desc = dsa.paged_desc(self.codes, self.table, self.ctx, max_len, scale=self.scale)

    def slots(self, seq, pos):
        seq, pos = torch.as_tensor(seq).long().cuda(), torch.as_tensor(pos).long().cuda()
        return self.table.long()[seq, pos // 64] * 64 + pos % 64


def check(latent, codes, scale, slots, kv, w, key, pos, freqs, half, key_half, rot0, m):
    """Flat caches: the named slots hold the rows, every other slot its pattern."""
    rows, k = oracle.cache_rows(f64(kv), f64(w), EPS, f64(key), pos, freqs.cpu().numpy(), half, key_half, rot0, m)
    a = np.abs(f64(kv)[:, 512:])
    both = np.tile(a[:, :32] + a[:, 32:], 2) if half else np.repeat(a[:, 0::2] + a[:, 1::2], 2, axis=1)
    bound = np.abs(rows) * 2.0 ** -8 * (1 + 2.0 ** -9) + np.concatenate([np.abs(rows[:, :512]) * 2.0 ** -18, m * 2.0 ** -20 * both], 1)
    err = np.abs(f64(latent[slots]) - rows)
    assert np.all(err <= bound), ("latent", np.argwhere(err > bound)[0])
    ktol = m * 2.0 ** -19 * 2 * np.abs(f64(key)).max(1)
    want = np.abs(k).max(1) / 448
    s = f64(scale[slots])
    assert np.all(np.abs(s - want) <= want * 2.0 ** -23 + ktol / 448), "scale"
    got = oracle.decode_e4m3(codes[slots].cpu().numpy()) * s[:, None]
    assert np.all(np.abs(got - k) <= np.maximum(np.abs(k) * 2.0 ** -4, s[:, None] * 2.0 ** -10) * (1 + 2.0 ** -10) + ktol[:, None]), "codes"
    rest = torch.ones(latent.shape[0], dtype=torch.bool, device="cuda")
    rest[slots] = False
    assert (latent[rest] == 7).all() and (codes[rest] == 0x55).all() and (scale[rest] == 5).all(), "other slots were written"


@pytest.mark.parametrize("rows", [1, 3, 64, 301])
@pytest.mark.parametrize("d_I", [64, 128])
@pytest.mark.parametrize("half,key_half", [(False, True), (True, False), (False, False), (True, True)])
def test_paged(rows, d_I, half, key_half):
    B = 3
    c = Caches(B, 9, d_I)
    kv, key, w = rnd((rows, 576), 1), rnd((rows, d_I), 2), 1 + 0.1 * rnd((512,), 3)
    g = torch.Generator().manual_seed(rows)
    flat = torch.randperm(B * 9 * 64, generator=g)[:rows]
    seq, pos = (flat // (9 * 64)).int(), (flat % (9 * 64)).int()
    freqs, m = dsa.dsa_rope_frequencies(64, 10000.0, dsa.DSA_ROPE_YARN, 40.0, 4096.0)
    freqs, rot0 = freqs.cuda(), 0 if rows % 2 else d_I - 64
    dsa.dsa_cache_append(kv, w, EPS, key, seq.cuda(), pos.cuda(), freqs, c.lat_desc, c.key_desc, ROPE[half], ROPE[key_half], rot0, m)
    assert dsa.dsa_device_error() == 0
    check(c.latent.flatten(0, 1), c.codes.flatten(0, 1), c.scale.flatten(), c.slots(seq, pos), kv, w, key, pos.numpy(), freqs, half,
          key_half, rot0, m)


def test_contiguous_and_a_rotated_range_inside_the_key():
    lens = [5, 0, 70, 1]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    T = sum(lens)
    latent = torch.full((T, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    codes, scale = torch.full((T, 128), 0x55, dtype=torch.uint8, device="cuda"), torch.full((T,), 5.0, device="cuda")
    seq = torch.tensor([0] * 4 + [2] * 70 + [3], dtype=torch.int32)
    pos = torch.tensor(list(range(4)) + list(range(70)) + [0], dtype=torch.int32)
    kv, key, w = rnd((75, 600), 1)[:, :576], rnd((75, 140), 2)[:, :128], rnd((512,), 3)  # strided rows
    freqs = dsa.dsa_rope_frequencies(64, 10000.0)[0].cuda()
    dsa.dsa_cache_append(kv, w, EPS, key, seq.cuda(), pos.cuda(), freqs, dsa.contiguous_desc(latent, cu, 70),
                         dsa.contiguous_desc(codes, cu, 70, scale=scale), key_rot_offset=22)
    assert dsa.dsa_device_error() == 0
    check(latent, codes, scale, cu.long()[seq.long().cuda()] + pos.long().cuda(), kv, w, key, pos.numpy(), freqs, False, True, 22, 1.0)


def test_one_token_per_sequence_without_a_row_map():
    c = Caches(70, 2, 128)
    kv, key, w = rnd((70, 576), 1), rnd((70, 128), 2), rnd((512,), 3)
    pos = torch.arange(70, dtype=torch.int32) + 30
    freqs = dsa.dsa_rope_frequencies(64, 10000.0)[0].cuda()
    dsa.dsa_cache_append(kv, w, EPS, key, None, pos.cuda(), freqs, c.lat_desc, c.key_desc)
    assert dsa.dsa_device_error() == 0
    check(c.latent.flatten(0, 1), c.codes.flatten(0, 1), c.scale.flatten(), c.slots(range(70), pos), kv, w, key, pos.numpy(), freqs,
          False, True, 0, 1.0)


def test_padding_and_rows_outside_the_caches_are_skipped():
    c = Caches(2, 3, 128)
    c.table[1, 1], c.table[1, 2] = -1, c.latent.shape[0]
    seq = torch.tensor([0, -1, 1, 1, 1, 0, 0, 2, -2, 1], dtype=torch.int32)
    pos = torch.tensor([5, 5, 0, 64, 128, 192, -1, 0, 0, 150], dtype=torch.int32)
    kv, key, w = rnd((10, 576), 1), rnd((10, 128), 2), rnd((512,), 3)
    freqs = dsa.dsa_rope_frequencies(64, 10000.0)[0].cuda()
    good = [0, 2]

    def go(rows, max_len=192):
        c.describe(max_len)
        r = torch.tensor(rows)
        dsa.dsa_cache_append(kv[r].contiguous(), w, EPS, key[r].contiguous(), seq[r].cuda(), pos[r].cuda(), freqs, c.lat_desc, c.key_desc)
        return dsa.dsa_device_error()

    assert go([0, 1, 2]) == 0                      # a padding row is no error
    for bad in range(3, 10):
        assert go([bad]) == dsa.DSA_ERR_DEVICE_CHECK, bad
    assert go([0], max_len=5) == dsa.DSA_ERR_DEVICE_CHECK  # position 5 of a cache of 5
    assert go(list(range(10))) == dsa.DSA_ERR_DEVICE_CHECK and dsa.dsa_device_error() == 0
    check(c.latent.flatten(0, 1), c.codes.flatten(0, 1), c.scale.flatten(), c.slots(seq[good], pos[good]), kv[good], w, key[good],
          pos[good].numpy(), freqs, False, True, 0, 1.0)


def test_either_half_alone():
    kv, key, w = rnd((3, 576), 1), rnd((3, 128), 2), rnd((512,), 3)
    seq, pos = torch.tensor([0, 0, 1], dtype=torch.int32).cuda(), torch.tensor([3, 4, 70], dtype=torch.int32).cuda()
    freqs = dsa.dsa_rope_frequencies(64, 10000.0)[0].cuda()
    a, b, d = Caches(2, 3, 128), Caches(2, 3, 128), Caches(2, 3, 128)
    dsa.dsa_cache_append(kv, w, EPS, key, seq, pos, freqs, a.lat_desc, a.key_desc)
    dsa.dsa_cache_append(kv, w, EPS, None, seq, pos, freqs, b.lat_desc, None)
    dsa.dsa_cache_append(None, None, 0.0, key, seq, pos, freqs, None, d.key_desc)
    assert torch.equal(a.latent, b.latent) and torch.equal(a.codes, d.codes) and torch.equal(a.scale, d.scale)
    assert (b.codes == 0x55).all() and (d.latent == 7).all()


def test_zero_nan_and_infinite_rows():
    kv, key, w = rnd((4, 576), 1), rnd((4, 128), 2), torch.ones(512, device="cuda").bfloat16()
    kv[0], key[0] = 0, 0
    kv[1, 10], key[1, 100] = float("nan"), float("nan")
    key[2, 100] = float("inf")
    c = Caches(4, 1, 128)
    freqs = dsa.dsa_rope_frequencies(64, 10000.0)[0].cuda()
    dsa.dsa_cache_append(kv, w, EPS, key, None, torch.full((4,), 9, dtype=torch.int32, device="cuda"), freqs, c.lat_desc, c.key_desc)
    at = c.slots(range(4), [9] * 4)
    lat, codes, scale = c.latent.flatten(0, 1)[at], c.codes.flatten(0, 1)[at], c.scale.flatten()[at]
    # a zero turned by a negative cosine is -0.0, whose code is 0x80: both codes stand for zero
    assert (lat[0] == 0).all() and (codes[0] & 0x7F == 0).all() and scale[0] == 1
    assert lat[1, :512].isnan().all() and lat[1, 512:].isfinite().all()
    assert codes[1, 100] & 0x7F == 0x7F and (codes[1, :100] & 0x7F != 0x7F).all() and scale[1].isfinite()
    assert scale[2].isinf() and lat[2].isfinite().all() and lat[3].isfinite().all()  # as dsa_quantize_fp8 gives


def test_slots_past_2_31_elements_of_a_pool():
    pages = 60000  # 60000 * 64 * 576 = 2.2e9
    latent = torch.zeros((pages, 64, 576), dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[0, pages - 1, 58300]], dtype=torch.int32, device="cuda")
    ctx = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv, w = rnd((3, 576), 1), rnd((512,), 2)
    pos = torch.tensor([63, 64, 191], dtype=torch.int32, device="cuda")
    freqs = dsa.dsa_rope_frequencies(64, 10000.0)[0].cuda()
    dsa.dsa_cache_append(kv, w, EPS, None, torch.zeros(3, dtype=torch.int32, device="cuda"), pos, freqs,
                         dsa.paged_desc(latent, table, ctx, 192), None)
    assert dsa.dsa_device_error() == 0
    small = Caches(1, 3, 128)
    dsa.dsa_cache_append(kv, w, EPS, None, torch.zeros(3, dtype=torch.int32, device="cuda"), pos, freqs, small.lat_desc, None)
    want = small.latent.flatten(0, 1)[small.slots([0, 0, 0], pos.cpu())]
    assert torch.equal(latent[0, 63], want[0]) and torch.equal(latent[pages - 1, 0], want[1]) and torch.equal(latent[58300, 63], want[2])
    assert (latent[1:58300] == 0).all()


def test_captured_steps_write_where_the_positions_say():
    c = Caches(4, 2, 128)
    kv, key, w = rnd((4, 576), 1), rnd((4, 128), 2), rnd((512,), 3)
    pos = torch.tensor([0, 10, 63, 100], dtype=torch.int32, device="cuda")
    freqs = dsa.dsa_rope_frequencies(64, 10000.0)[0].cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.dsa_cache_append(kv, w, EPS, key, None, pos, freqs, c.lat_desc, c.key_desc)
        pos.add_(1)
    start = pos.cpu().numpy().copy()
    for _ in range(3):
        g.replay()
    other = Caches(4, 2, 128)
    for i in range(3):
        at = torch.tensor(start + i, device="cuda")
        dsa.dsa_cache_append(kv, w, EPS, key, None, at, freqs, other.lat_desc, other.key_desc)
    assert dsa.dsa_device_error() == 0 and (pos.cpu().numpy() == start + 3).all()
    assert torch.equal(c.latent, other.latent) and torch.equal(c.codes, other.codes) and torch.equal(c.scale, other.scale)


def test_wrapper_refusals():
    c, other = Caches(2, 2, 128), Caches(3, 2, 64)
    kv, key, w = rnd((2, 576), 1), rnd((2, 128), 2), rnd((512,), 3)
    pos, freqs = torch.zeros(2, dtype=torch.int32, device="cuda"), dsa.dsa_rope_frequencies(64, 10000.0)[0].cuda()
    ok = dict(kv=kv, kv_weight=w, eps=EPS, key=key, seq=None, positions=pos, freqs=freqs, latent=c.lat_desc, keys=c.key_desc)
    for kw in (dict(kv=kv.float()), dict(kv=kv[:1]), dict(key=key[:1]), dict(key=key[:, :64]), dict(positions=pos.long()),
               dict(seq=pos[:1]), dict(freqs=freqs.float()), dict(freqs=freqs.cpu()), dict(kv_weight=w[:100]), dict(keys=other.key_desc),
               dict(latent=c.key_desc), dict(keys=c.lat_desc), dict(latent=other.lat_desc)):
        with pytest.raises(ValueError):
            dsa.dsa_cache_append(**{**ok, **kw})
    wide_table = dsa.paged_desc(c.latent, c.table.long(), c.ctx, 128)
    half_scale = dsa.paged_desc(c.codes, c.table, c.ctx, 128, scale=c.scale.half())
    for kw in (dict(latent=wide_table), dict(keys=half_scale), dict(latent=dsa.paged_desc(c.latent, c.table.cpu(), c.ctx, 128))):
        with pytest.raises(ValueError):
            dsa.dsa_cache_append(**{**ok, **kw})
    for kw in (dict(kv=None), dict(keys=None), dict(key_rot_offset=66), dict(kv_weight=None), dict(layout=5)):
        with pytest.raises(dsa.DSAError):
            dsa.dsa_cache_append(**{**ok, **kw})
    assert (c.latent == 7).all()


def test_the_stride_of_a_single_row_does_not_matter():
    c = Caches(2, 2, 128)
    kv, key, w = rnd((1, 577), 1)[:, :576], rnd((1, 129), 2)[:, :128], rnd((512,), 3)
    assert kv.stride(0) == 577 and key.stride(0) == 129
    pos, freqs = torch.tensor([70], dtype=torch.int32), dsa.dsa_rope_frequencies(64, 10000.0)[0].cuda()
    dsa.dsa_cache_append(kv, w, EPS, key, torch.ones(1, dtype=torch.int32, device="cuda"), pos.cuda(), freqs, c.lat_desc, c.key_desc)
    assert dsa.dsa_device_error() == 0
    check(c.latent.flatten(0, 1), c.codes.flatten(0, 1), c.scale.flatten(), c.slots([1], pos), kv, w, key, pos.numpy(), freqs, False,
          True, 0, 1.0)
    many_kv, many_key = rnd((2, 577), 1)[:, :576], rnd((2, 129), 2)[:, :128]  # of two rows it does
    pos2, seq2 = torch.tensor([3, 4], dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    for kw in ((many_kv, None), (None, many_key)):
        with pytest.raises(dsa.DSAError):
            dsa.dsa_cache_append(kw[0], w if kw[0] is not None else None, EPS, kw[1], seq2, pos2, freqs,
                                 c.lat_desc if kw[0] is not None else None, c.key_desc if kw[1] is not None else None)
