"""Host side of the operators around the caches: every refusal that needs no GPU (the calls return
before a launch), the frequency tables, the workspace rules."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import sparse_attention_09_b200 as dsa

INVALID, UNSUPPORTED, SMALL, OK = dsa.DSA_ERR_INVALID_ARGUMENT, dsa.DSA_ERR_UNSUPPORTED, dsa.DSA_ERR_WORKSPACE_TOO_SMALL, dsa.DSA_OK
A = 4096  # an aligned address that no refused call reads


def norm(**kw):
    a = dict(x=A, ld_x=64, res=None, ld_res=0, w=A, rows=4, cols=64, dtype=0, eps=1e-6, y=2 * A, ld_y=64, ro=None, ld_ro=0, codes=None,
             scale=None, group=0, rstd=None)
    a.update(kw)
    return dsa._lib.dsa_rmsnorm(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0, x=None), OK), (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(x=None), INVALID),
    (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(codes=A), INVALID), (dict(scale=A), INVALID),
    (dict(codes=A, scale=A, group=64), INVALID), (dict(ld_x=-1), INVALID), (dict(y=A, x=A, ld_x=128), INVALID), (dict(y=A, res=A, ld_res=0), INVALID),
    (dict(ro=A, ld_ro=64, y=A), INVALID), (dict(ld_y=63), INVALID), (dict(res=A, ld_res=-8), INVALID),
    (dict(ro=A, ld_ro=8), INVALID), (dict(x=A + 1), INVALID), (dict(dtype=2, x=A + 2), INVALID), (dict(codes=A, scale=A + 2), INVALID),
    (dict(rows=1 << 31), UNSUPPORTED)])
def test_rmsnorm_refusals(kw, want):
    assert norm(**kw) == want


def norm_bwd(**kw):
    a = dict(dy=A, ld_dy=64, h=A, ld_h=64, w=A, rstd=A, dres=None, ld_dres=0, rows=4, cols=64, dtype=0, dh=A, ld_dh=64, dw=A, ws=A,
             size=1 << 20)
    a.update(kw)
    return dsa._lib.dsa_rmsnorm_backward(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(dtype=7), INVALID), (dict(dy=None), INVALID), (dict(h=None), INVALID),
    (dict(w=None), INVALID), (dict(rstd=None), INVALID), (dict(dh=None), INVALID), (dict(dw=None), INVALID), (dict(ws=None), INVALID),
    (dict(ws=A + 8), INVALID), (dict(ld_dy=-1), INVALID), (dict(ld_h=-1), INVALID), (dict(ld_dy=128), INVALID), (dict(ld_dh=1), INVALID),
    (dict(dres=A, ld_dres=-3), INVALID), (dict(dh=2 * A, dres=2 * A, ld_dres=0), INVALID), (dict(h=A + 1), INVALID), (dict(size=4 * 64 * 4 - 1), SMALL), (dict(rows=1 << 31), UNSUPPORTED)])
def test_rmsnorm_backward_refusals(kw, want):
    assert norm_bwd(**kw) == want


def test_rmsnorm_backward_workspace_grows_to_a_limit():
    f = dsa.dsa_rmsnorm_backward_workspace_size
    assert f(0, 64) == 0 and f(4, 0) == 0
    assert f(4, 64) >= 4 * 64 * 4 and f(10 ** 6, 64) == f(10 ** 9, 64)


def rope(**kw):
    a = dict(x=A, xr=512, xh=128, out=2 * A, orow=512, oh=128, rows=3, heads=4, dim=128, off=0, rot=64, layout=0, dtype=0, pos=A,
             freqs=A, m=1.0, t=0)
    a.update(kw)
    return dsa._lib.dsa_rope(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0, x=None), OK), (dict(heads=0, x=None), OK), (dict(rows=-1), INVALID), (dict(heads=-1), INVALID), (dict(dim=0), INVALID),
    (dict(rot=63), INVALID), (dict(rot=0), INVALID), (dict(off=65), INVALID), (dict(off=-1), INVALID), (dict(rot=130), INVALID),
    (dict(layout=2), INVALID), (dict(dtype=3), INVALID), (dict(m=float("inf")), INVALID), (dict(x=None), INVALID), (dict(out=None), INVALID),
    (dict(pos=None), INVALID), (dict(freqs=None), INVALID), (dict(freqs=A + 4), INVALID), (dict(x=A + 1), INVALID), (dict(xh=-1), INVALID),
    (dict(oh=127), INVALID), (dict(orow=100), INVALID), (dict(orow=500), INVALID), (dict(orow=128, oh=128), INVALID), (dict(xr=-8), INVALID), (dict(out=A, oh=256), INVALID), (dict(out=A, orow=1024), INVALID),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(dim=2048, xh=2048, oh=2048, xr=8192, orow=8192, rot=1026), UNSUPPORTED)])
def test_rope_refusals(kw, want):
    assert rope(**kw) == want


@pytest.mark.parametrize("scaling,name", [(0, "plain"), (1, "linear"), (2, "ntk"), (3, "yarn")])
@pytest.mark.parametrize("rot,theta,factor,ctx", [(64, 10000.0, 40.0, 4096.0), (4, 500.0, 1.0, 100.0), (128, 1e6, 3.5, 32768.0)])
def test_rope_frequencies_match_the_oracle(scaling, name, rot, theta, factor, ctx):
    got, m = dsa.dsa_rope_frequencies(rot, theta, scaling, factor, ctx)
    want, wm = oracle.rope_frequencies(rot, theta, name, factor, ctx)
    assert got.dtype == torch.float64 and got.shape == (rot // 2,)
    assert np.allclose(got.numpy(), want, rtol=1e-14, atol=0) and np.isclose(m, wm, rtol=2.0 ** -24)


@pytest.mark.parametrize("args", [(0, 1e4), (7, 1e4), (64, 1.0), (64, float("nan")), (64, 1e4, 4), (64, 1e4, -1), (64, 1e4, 1, 0.5),
                                  (2, 1e4, 2, 2.0), (64, 1e4, 3, 2.0, 0.0), (64, 1e4, 3, 2.0, 4096.0, 1.0, 2.0),
                                  (64, 1e4, 3, 2.0, 4096.0, 32.0, 0.0), (64, 1e4, 3, float("inf"), 4096.0)])
def test_rope_frequencies_refusals(args):
    with pytest.raises(dsa.DSAError) as e:
        dsa.dsa_rope_frequencies(*args)
    assert e.value.status == INVALID


def test_rope_frequencies_read_only_what_their_scaling_needs():
    assert dsa.dsa_rope_frequencies(64, 1e4, dsa.DSA_ROPE_PLAIN, factor=0.0)[1] == 1.0
    dsa.dsa_rope_frequencies(64, 1e4, dsa.DSA_ROPE_LINEAR, 2.0, original_ctx=-1.0, beta_slow=0.0)


def paged(**kw):
    a = dict(kind=dsa.DSA_KV_PAGED, data=A, scale=A, cu=None, table=A, ctx=A, total=0, max_seqlen=640, blocks=20, size=64, per=10)
    a.update(kw)
    return dsa.KVDesc(*a.values())


def flat(**kw):
    return paged(**{**dict(kind=dsa.DSA_KV_CONTIGUOUS, cu=A, table=None, ctx=None, total=100, max_seqlen=100, blocks=0, size=0, per=0), **kw})


def append(latent=paged(), keys=paged(), **kw):
    a = dict(kv=A, ld_kv=576, w=A, eps=1e-6, key=A, ld_key=128, d_i=128, seq=A, pos=A, rows=2, B=2, freqs=A, m=1.0, layout=0, key_layout=1,
             rot0=0)
    a.update(kw)
    ref = lambda d: None if d is None else ctypes.byref(d)  # noqa: E731
    return dsa._lib.dsa_cache_append(*a.values(), ref(latent), ref(keys), None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), OK), (dict(rows=-1), INVALID), (dict(B=0), INVALID), (dict(kv=None), INVALID), (dict(key=None), INVALID),
    (dict(latent=None), INVALID), (dict(keys=None), INVALID), (dict(kv=None, latent=None, key=None, keys=None), INVALID),
    (dict(w=None), INVALID), (dict(pos=None), INVALID), (dict(freqs=None), INVALID), (dict(freqs=A + 4), INVALID), (dict(kv=A + 8), INVALID),
    (dict(ld_kv=580), INVALID), (dict(ld_kv=568), INVALID), (dict(key=A + 2), INVALID), (dict(ld_key=129), INVALID), (dict(ld_key=64), INVALID),
    (dict(d_i=96), UNSUPPORTED), (dict(rot0=1), INVALID), (dict(rot0=66), INVALID), (dict(rot0=-2), INVALID), (dict(d_i=64, rot0=2), INVALID),
    (dict(layout=2), INVALID), (dict(key_layout=2), INVALID), (dict(eps=-1.0), INVALID), (dict(m=float("nan")), INVALID),
    (dict(latent=paged(size=32)), UNSUPPORTED), (dict(latent=paged(data=None)), INVALID), (dict(latent=paged(data=A + 8)), INVALID),
    (dict(keys=paged(scale=None)), INVALID), (dict(keys=paged(data=A + 1)), INVALID), (dict(keys=paged(table=None)), INVALID),
    (dict(latent=paged(blocks=0)), INVALID), (dict(latent=paged(max_seqlen=0)), INVALID), (dict(latent=flat(cu=None)), INVALID),
    (dict(latent=flat(total=0)), INVALID), (dict(latent=paged(kind=5)), INVALID), (dict(rows=1 << 31), UNSUPPORTED)])
def test_cache_append_refusals(kw, want):
    assert append(**kw) == want


def window_prefill(latent=flat(), **kw):
    a = dict(q=A, latent=ctypes.byref(latent), B=1, H=128, window=8, sinks=0, sm=0.04, out=A, lse=A)
    a.update(kw)
    return dsa._lib.dsa_window_mla_prefill(*a.values(), None)


def window_decode(latent=paged(), **kw):
    a = dict(q=A, latent=ctypes.byref(latent), B=2, H=128, window=1000, sinks=0, sm=0.04, out=A, lse=A, ws=A, size=1 << 30)
    a.update(kw)
    return dsa._lib.dsa_window_mla_decode(*a.values(), None)


COMMON = [(dict(q=None), INVALID), (dict(out=None), INVALID), (dict(latent=None), INVALID), (dict(B=0), INVALID), (dict(H=0), UNSUPPORTED),
          (dict(H=129), UNSUPPORTED), (dict(window=0), INVALID), (dict(sinks=-1), INVALID), (dict(sm=-0.1), INVALID), (dict(sm=0.0), INVALID),
          (dict(sm=float("nan")), INVALID), (dict(sm=float("inf")), INVALID), (dict(q=A + 8), INVALID), (dict(out=A + 8), INVALID),
          (dict(lse=A + 2), INVALID)]


@pytest.mark.parametrize("kw,want", COMMON)
def test_window_refusals(kw, want):
    for call in (window_prefill, window_decode):
        if "latent" in kw:
            assert dsa._lib.dsa_window_mla_prefill(A, None, 1, 128, 8, 0, 0.04, A, A, None) == want
            assert dsa._lib.dsa_window_mla_decode(A, None, 1, 128, 8, 0, 0.04, A, A, A, 1 << 30, None) == want
        else:
            assert call(**kw) == want


def test_window_descriptor_refusals():
    assert window_prefill(paged()) == INVALID and window_decode(flat()) == INVALID
    assert window_prefill(flat(data=A + 8)) == INVALID and window_prefill(flat(total=0)) == INVALID
    assert window_prefill(flat(max_seqlen=0)) == INVALID and window_prefill(flat(total=1 << 25)) == UNSUPPORTED
    assert window_decode(paged(size=32)) == UNSUPPORTED and window_decode(paged(max_seqlen=641)) == INVALID
    assert window_decode(paged(table=None)) == INVALID and window_decode(paged(ctx=None)) == INVALID
    assert window_decode(paged(blocks=1 << 25)) == UNSUPPORTED


def test_window_decode_workspace():
    # chunks of 128 keys are shared out when the even share (a query counting 2 beside its own), an eighth
    # of it and 8 come to less than rounds of whole sequences over 74 clusters
    f = dsa.dsa_window_mla_workspace_size
    assert f(0, 128, 8, 0, 100) == 0 and f(4, 128, 0, 0, 100) == 0 and f(4, 128, 8, 0, 0) == 0

    def expected(B, H, window, sinks, ctx):
        chunks = -(-min(ctx, window + sinks) // 128)
        share = B * (chunks + 2) // 74
        if B > 1024 or chunks < 2 or not share + share // 8 + 8 < -(-B // 74) * (chunks + 2):
            return 0
        up = lambda n: -(-n // 256) * 256  # noqa: E731
        return up(B * 8) + up(148 * H * 512 * 4) + up(148 * H * 8)

    for B in (1, 2, 37, 63, 64, 73, 74, 75, 80, 148, 1024, 1025):
        for window, sinks, ctx in ((64, 0, 10 ** 5), (100, 30, 10 ** 5), (512, 4, 10 ** 5), (4096, 0, 9000), (2 ** 31 - 1, 2 ** 31 - 1, 131072)):
            assert f(B, 128, window, sinks, ctx) == expected(B, 128, window, sinks, ctx), (B, window)
    assert f(1, 128, 64, 0, 100000) == 0 and f(3, 128, 2 ** 31 - 1, 0, 131072) > 0 and f(74, 128, 4096, 0, 131072) == 0
    d = paged(max_seqlen=6400, per=100)
    need = f(2, 128, 5000, 0, 6400)
    assert need > 0
    assert window_decode(d, window=5000, size=need - 1) == SMALL and window_decode(d, window=5000, ws=None) == INVALID
    assert window_decode(d, window=5000, ws=A + 128) == INVALID


def test_wrappers_refuse_tensors_they_cannot_pass_on():
    x, w = torch.zeros(4, 8), torch.zeros(8)
    pos, freqs = torch.zeros(4, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError):
        dsa.dsa_rmsnorm(x, w, 1e-6, y=x)                                     # not on a GPU
    with pytest.raises(ValueError):
        dsa.dsa_rmsnorm_backward(x, x, w, w, x, w, w)
    with pytest.raises(ValueError):
        dsa.dsa_rope(x.view(4, 1, 8), pos, freqs, x.view(4, 1, 8), 0, 8)
    with pytest.raises(ValueError):
        dsa.dsa_cache_append(None, None, 0.0, x.bfloat16(), None, pos, freqs, None, None)
    lat = dsa.contiguous_desc(torch.zeros(4, 576, dtype=torch.bfloat16), torch.tensor([0, 4], dtype=torch.int32), 4)
    q, out = torch.zeros(4, 16, 576, dtype=torch.bfloat16), torch.zeros(4, 16, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dsa.dsa_window_mla_prefill(q, lat, 1, 16, 4, 0, 0.04, out)
    with pytest.raises(ValueError):
        dsa.dsa_window_mla_decode(q, lat, 4, 16, 4, 0, 0.04, out)


def test_wrappers_refuse_what_is_no_tensor_or_does_not_fit():
    x, w = torch.zeros(4, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="x must be a tensor"):
        dsa.dsa_rmsnorm([1.0], w, 1e-6, y=x)
    with pytest.raises(ValueError, match="x must be a tensor"):
        dsa.dsa_rope(None, None, None, x, 0, 8)
    with pytest.raises(ValueError, match="current CUDA device"):
        dsa.dsa_rmsnorm(x, w, "no number", y=x)  # the tensors are looked at first
    with pytest.raises(ValueError, match="takes 10 arguments"):
        dsa._marshal.rmsnorm(x, w)
    lat = dsa.contiguous_desc(torch.zeros(4, 576, dtype=torch.bfloat16), torch.tensor([0, 4], dtype=torch.int32), 4)
    q, out = torch.zeros(4, 16, 576, dtype=torch.bfloat16), torch.zeros(4, 16, 512, dtype=torch.bfloat16)
    for B in (0, 2, -1):
        with pytest.raises(ValueError, match="sequences"):
            dsa.dsa_window_mla_prefill(q, lat, B, 16, 4, 0, 0.04, out)
    bad = dsa.contiguous_desc(torch.zeros(4, 576, dtype=torch.bfloat16), torch.tensor([0, 4]), 4)
    with pytest.raises(ValueError, match="int32"):
        dsa.dsa_window_mla_prefill(q, bad, 1, 16, 4, 0, 0.04, out)
    with pytest.raises(ValueError, match="rows of 576"):
        dsa.dsa_window_mla_prefill(q, dsa.contiguous_desc(torch.zeros(4, 576), lat._refs[2], 4), 1, 16, 4, 0, 0.04, out)


@pytest.mark.parametrize("data,table,ctx", [
    ((10, 576), (2, 4), (2,)),          # no page dimension: its 576 would be taken for the page size
    ((10, 64, 2, 576), (2, 4), (2,)),   # two rows per slot
    ((10, 64, 576), (2, 4), (1,)),      # fewer lengths than sequences
    ((10, 64, 576), (2, 4), (3,)),
    ((10, 64, 576), (0, 4), (0,)),
    ((10, 64, 576), (2, 4, 2), (2,))])
def test_wrappers_refuse_descriptors_that_do_not_fit_their_tensors(data, table, ctx):
    desc = dsa.paged_desc(torch.zeros(data, dtype=torch.bfloat16), torch.zeros(table, dtype=torch.int32),
                          torch.zeros(ctx, dtype=torch.int32), 256)
    B = table[0]
    q, out = torch.zeros(B, 16, 576, dtype=torch.bfloat16), torch.zeros(B, 16, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="latent"):
        dsa.dsa_window_mla_decode(q, desc, B, 16, 8, 0, 0.04, out)
    with pytest.raises(ValueError, match="latent"):
        dsa.dsa_cache_append(torch.zeros(B, 576), None, 1e-6, None, None, torch.zeros(B, dtype=torch.int32), None, desc, None)


def test_wrappers_refuse_packed_lengths_of_another_rank():
    for cu in ((2, 2), (1,)):
        desc = dsa.contiguous_desc(torch.zeros(4, 576, dtype=torch.bfloat16), torch.zeros(cu, dtype=torch.int32), 4)
        with pytest.raises(ValueError, match="latent"):
            dsa.dsa_window_mla_prefill(torch.zeros(4, 16, 576), desc, desc.batch, 16, 8, 0, 0.04, torch.zeros(4, 16, 512))


def test_wrappers_take_a_head_dimension_of_one():
    """[blocks, 64, 1, 576], as caches with a head dimension are laid out: the rows are the same."""
    desc = dsa.paged_desc(torch.zeros(3, 64, 1, 576, dtype=torch.bfloat16), torch.zeros(2, 4, dtype=torch.int32),
                          torch.zeros(2, dtype=torch.int32), 256)
    with pytest.raises(ValueError, match="current CUDA device"):  # refused for being on the CPU, not for its shape
        dsa.dsa_window_mla_decode(torch.zeros(2, 16, 576), desc, 2, 16, 8, 0, 0.04, torch.zeros(2, 16, 512))


def test_rows_too_wide_for_32_bit_columns():
    wide = 2 ** 31 - 512  # a step of 1024 past the last column leaves 32 bits
    assert norm(cols=wide, ld_x=wide, ld_y=wide) == UNSUPPORTED
    assert norm_bwd(cols=wide, ld_dy=wide, ld_h=wide, ld_dh=wide, size=1 << 62) == UNSUPPORTED
    assert rope(heads=1, dim=wide, xr=wide, orow=wide) == UNSUPPORTED
    assert rope(heads=2 ** 20, dim=2 ** 10 + 8, xh=2048, oh=2048, xr=2 ** 31, orow=2 ** 31) == UNSUPPORTED


def test_contexts_too_long_for_32_bit_entries():
    assert window_decode(paged(max_seqlen=2 ** 30 + 1, per=2 ** 25)) == UNSUPPORTED


def test_rmsnorm_backward_workspace_serves_smaller_calls():
    """One workspace for the widest layer and the longest batch serves all others; without the rule 65536 rows of 5120 columns
    asked for 3.03 MB and of 4096 columns for 4.85 MB."""
    f = dsa.dsa_rmsnorm_backward_workspace_size
    for rows in (1, 37, 148, 149, 1000, 2367, 2368, 65536):
        sizes = [f(rows, c) for c in range(1, 12300)]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])), rows
        # what a call of these sizes writes: a row of partial sums for each of min(rows, 148 x (16 KB / row, 1 to 16)) CTAs
        own = [min(rows, 148 * min(max(16384 // (2 * c), 1), 16)) * c * 4 for c in range(1, 12300)]
        most = np.maximum.accumulate(own)
        assert all(s == -(-int(m) // 256) * 256 for s, m in zip(sizes, most)), rows
    for cols in (8, 500, 4096, 5120, 20000):
        sizes = [f(r, cols) for r in list(range(1, 2500)) + [10 ** 6, 2 ** 31 - 1]]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])), cols


def test_window_workspace_limit_serves_smaller_batches():
    """The need of one call is not monotone (64 sequences none, 48 some); the limit covers every smaller call and is reached."""
    size, limit = dsa.dsa_window_mla_workspace_size, dsa.dsa_window_mla_workspace_limit
    assert size(64, 128, 4096, 16, 32768) == 0 and size(48, 128, 4096, 16, 32768) > 0
    assert limit(0, 128, 8, 0, 100) == 0 and limit(4, 128, 0, 0, 100) == 0 and limit(4, 0, 8, 0, 100) == 0 and limit(4, 128, 8, -1, 9) == 0
    for keys in list(range(1, 2000, 63)) + [767, 768, 769, 896, 897, 4112, 32768, 131072]:
        most, smaller = 0, limit(1, 128, keys, 0, 2 ** 30)
        for B in range(1, 1200):
            most = max(most, size(B, 128, keys, 0, 2 ** 30), size(B, 128, 2 ** 30, 0, keys))
            got = limit(B, 128, keys, 0, 2 ** 30)
            assert got == limit(B, 128, 2 ** 30, 5, keys) >= max(most, smaller) and (got == 0) == (most == 0), (B, keys)
            assert got - most <= B * 8 + 256  # the plan of the largest batch beside the parts of another
            smaller = got
        assert limit(64, 64, keys, 0, 2 ** 30) <= limit(64, 128, keys, 0, 2 ** 30) <= limit(64, 128, keys + 1, 0, 2 ** 30)
    d = paged(max_seqlen=32768, per=512)
    need = limit(64, 128, 4096, 16, 32768)
    for B in (1, 2, 40, 48):
        assert 0 < size(B, 128, 4096, 16, 32768) <= need
        assert window_decode(d, B=B, window=4096, sinks=16, size=size(64, 128, 4096, 16, 32768)) == SMALL


def test_sizes_beyond_their_integers_are_refused_and_not_cut():
    """A window of 2^31 for "everything" was cut to a negative one, for which no workspace is needed."""
    for f in (dsa.dsa_window_mla_workspace_size, dsa.dsa_window_mla_workspace_limit):
        assert f(3, 128, 2 ** 31 - 1, 0, 131072) > 0
        for args in ((3, 128, 2 ** 31, 0, 131072), (3, 128, 4096, 2 ** 32, 131072), (2 ** 32 + 3, 128, 4096, 0, 131072), (3, -2 ** 31 - 1, 4096, 0, 1),
                     (3, 128, 4096, 0, 2 ** 32 + 131072)):
            with pytest.raises(ValueError, match="32 bits"):
                f(*args)
    for args in ((4, 2 ** 32 + 64), (4, -2 ** 31 - 1)):
        with pytest.raises(ValueError, match="32 bits"):
            dsa.dsa_rmsnorm_backward_workspace_size(*args)
    with pytest.raises(ValueError, match="64 bits"):
        dsa.dsa_rmsnorm_backward_workspace_size(2 ** 64 + 4, 64)
    for args in ((-2 ** 32 + 64, 1e4), (64, 1e4, 2 ** 32)):  # the table of 2^31 and more dims itself is not asked for here
        with pytest.raises(ValueError, match="32 bits"):
            dsa.dsa_rope_frequencies(*args)


def test_wrappers_refuse_what_is_no_descriptor_or_tensor_by_value_error():
    q, out, pos = torch.zeros(2, 16, 576, dtype=torch.bfloat16), torch.zeros(2, 16, 512, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    lat = dsa.contiguous_desc(torch.zeros(2, 576, dtype=torch.bfloat16), torch.tensor([0, 2], dtype=torch.int32), 2)
    for call in (dsa.dsa_window_mla_prefill, dsa.dsa_window_mla_decode):
        for desc in (None, q, lat.struct):
            with pytest.raises(ValueError, match="latent must be"):
                call(q, desc, 1, 16, 8, 0, 0.04, out)
        with pytest.raises(ValueError, match="q must be a tensor"):
            call(None, lat, 1, 16, 8, 0, 0.04, out)
    for bad in (q, lat.struct, 3):
        with pytest.raises(ValueError, match="latent must be"):
            dsa.dsa_cache_append(q, None, 0.0, None, None, pos, None, bad, None)
        with pytest.raises(ValueError, match="keys must be"):
            dsa.dsa_cache_append(None, None, 0.0, pos, None, pos, None, None, bad)
    with pytest.raises(ValueError, match="positions must be a tensor"):
        dsa.dsa_cache_append(None, None, 0.0, None, None, None, None, lat, None)
    with pytest.raises(ValueError, match="key must be a tensor"):
        dsa.dsa_cache_append(None, None, 0.0, [1.0], None, pos, None, None, lat)
