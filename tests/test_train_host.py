"""Host-side checks of a training step's operators: the C entries refuse bad arguments before any CUDA work, the Python
entries refuse wrong types and devices.  Runs without a GPU."""
import ctypes
import math

import pytest
import torch

import gated_deltanet_chunked_chunk_gb300 as gdn
from gated_deltanet_chunked_chunk_gb300 import build as gbuild

F = ctypes.c_void_p(4096)  # never dereferenced: every call below is refused, or has nothing to do
ODD = ctypes.c_void_p(4098)
BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdn.load_library()


def _call(lib, name, order, defaults, kw):
    a = dict(defaults)
    a.update(kw)
    return getattr(lib, name)(*[a[k] for k in order.split()])


SIZES = dict(cu=None, cu_k=None, N=1, Tq=256, Tk=256, HQ=8, HK=2, D=128, causal=1, scale=-1.0, status=None, stream=None,
             q=F, ldq=1024, k=F, ldk=256, v=F, ldv=256)
FWD = "q ldq k ldk v ldv cu cu_k N Tq Tk HQ HK D causal scale o lse status stream"
BWD = "do q ldq k ldk v ldv o lse cu cu_k N Tq Tk HQ HK D causal scale dq dk dv ws bytes status stream"


def _fwd(lib, **kw):
    return _call(lib, "gdn_attention_fwd", FWD, dict(SIZES, o=F, lse=F), kw)


def _bwd(lib, **kw):
    return _call(lib, "gdn_attention_bwd", BWD, dict(SIZES, do=F, o=F, lse=F, dq=F, dk=F, dv=F, ws=F, bytes=1 << 40), kw)


BAD = [dict(N=-1), dict(Tq=-1), dict(Tk=-1), dict(HQ=0), dict(HK=0), dict(HQ=7), dict(D=0), dict(causal=2), dict(N=2), dict(cu_k=F),
       dict(cu=F, Tk=128), dict(q=None), dict(k=None), dict(v=None), dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(ldq=1016),
       dict(ldk=248), dict(ldv=248), dict(ldq=1028), dict(ldk=260), dict(ldv=258)]
TOO_MUCH = [dict(D=96), dict(D=256, ldq=2048, ldk=512, ldv=512), dict(N=65536, cu=F), dict(HQ=65536, HK=65536, ldq=1 << 23, ldk=1 << 23, ldv=1 << 23),
            dict(ldq=1 << 40)]


@pytest.mark.parametrize("kw", BAD + [dict(o=None), dict(lse=None), dict(o=ODD)])
def test_attention_fwd_refusals(lib, kw):
    assert _fwd(lib, **kw) == gdn.GDN_EINVAL


@pytest.mark.parametrize("kw", BAD + [dict(do=None), dict(o=None), dict(lse=None), dict(dq=None), dict(dk=None), dict(dv=None), dict(do=ODD),
                                      dict(dq=ODD), dict(dk=ODD), dict(dv=ODD), dict(ws=ODD)])
def test_attention_bwd_refusals(lib, kw):
    assert _bwd(lib, **kw) == gdn.GDN_EINVAL


@pytest.mark.parametrize("kw", TOO_MUCH)
def test_attention_sizes_that_are_not_supported(lib, kw):
    assert _fwd(lib, **kw) == gdn.GDN_EUNSUPPORTED
    assert _bwd(lib, **kw) == gdn.GDN_EUNSUPPORTED


def test_attention_workspace(lib):
    need = gdn.attention_bwd_workspace_size(1, 256, 256, 8, 2, 128)
    assert need > 0
    assert _bwd(lib, bytes=need - 1) == gdn.GDN_EWORKSPACE
    assert _bwd(lib, ws=None) == gdn.GDN_EWORKSPACE
    for bad in ((-1, 1, 1, 1, 1, 64), (1, -1, 1, 1, 1, 64), (1, 1, 1, 3, 2, 64), (1, 1, 1, 1, 1, 96), (65536, 1, 1, 1, 1, 64)):
        assert gdn.attention_bwd_workspace_size(*bad) == 0


def test_attention_without_rows(lib):
    assert _fwd(lib, Tq=0, q=None, o=None, lse=None) == gdn.GDN_OK
    nothing = dict(Tq=0, Tk=0, q=None, k=None, v=None, do=None, o=None, lse=None, dq=None, dk=None, dv=None, ws=None, bytes=0)
    assert _bwd(lib, **nothing) == gdn.GDN_OK


def _save(lib, **kw):
    return _call(lib, "gdn_act8_save", "x rows D x_rows x_stride codes scale stream",
                 dict(x=F, rows=4, D=128, x_rows=0, x_stride=0, codes=F, scale=F, stream=None), kw)


def _load(lib, **kw):
    return _call(lib, "gdn_act8_load", "codes scale rows D y stream", dict(codes=F, scale=F, rows=4, D=128, y=F, stream=None), kw)


@pytest.mark.parametrize("kw", [dict(x=None), dict(codes=None), dict(scale=None), dict(rows=-1), dict(D=0), dict(x_rows=-1)])
def test_act8_save_refusals(lib, kw):
    assert _save(lib, **kw) == gdn.GDN_EINVAL


@pytest.mark.parametrize("kw", [dict(codes=None), dict(scale=None), dict(y=None), dict(rows=-1), dict(D=0)])
def test_act8_load_refusals(lib, kw):
    assert _load(lib, **kw) == gdn.GDN_EINVAL


def test_act8_without_rows(lib):
    assert _save(lib, rows=0, x=None, codes=None, scale=None) == gdn.GDN_OK
    assert _load(lib, rows=0, codes=None, scale=None, y=None) == gdn.GDN_OK


def _norm(lib, **kw):
    order = ("x residual z weight res_scale eps activation rows D z_rows z_stride y h h_codes h_scale z_codes z_scale stream")
    return _call(lib, "gdn_norm_gate_save8", order, dict(
        x=F, residual=None, z=None, weight=F, res_scale=1.0, eps=1e-6, activation=0, rows=4, D=128, z_rows=0, z_stride=0, y=F, h=None,
        h_codes=F, h_scale=F, z_codes=None, z_scale=None, stream=None), kw)


def _norm_b(lib, **kw):
    order = ("dy h_codes h_scale z_codes z_scale dh weight res_scale eps activation rows D dx dresidual dz dweight ws bytes stream")
    return _call(lib, "gdn_norm_gate_bwd8", order, dict(
        dy=F, h_codes=F, h_scale=F, z_codes=None, z_scale=None, dh=None, weight=F, res_scale=1.0, eps=1e-6, activation=0, rows=4, D=128,
        dx=F, dresidual=None, dz=None, dweight=F, ws=F, bytes=1 << 30, stream=None), kw)


GATE = dict(activation=1, z=F, z_codes=F, z_scale=F)


@pytest.mark.parametrize("kw", [dict(x=None), dict(weight=None), dict(y=None), dict(h_codes=None), dict(h_scale=None), dict(D=0), dict(rows=-1),
                                dict(activation=3), dict(activation=1), dict(z=F), dict(GATE, z_codes=None), dict(GATE, z_scale=None),
                                dict(z_codes=F), dict(residual=F), dict(h=F), dict(eps=math.nan), dict(eps=-1.0), dict(GATE, z_rows=-1),
                                dict(GATE, z_rows=1, z_stride=132), dict(x=ODD), dict(y=ODD), dict(h_codes=ODD), dict(GATE, z=ODD),
                                dict(GATE, z_codes=ODD), dict(residual=ODD, h=F), dict(residual=F, h=ODD)])
def test_norm_gate_save8_refusals(lib, kw):
    assert _norm(lib, **kw) == gdn.GDN_EINVAL


@pytest.mark.parametrize("kw", [dict(dy=None), dict(h_codes=None), dict(h_scale=None), dict(weight=None), dict(dx=None), dict(dweight=None),
                                dict(D=0), dict(rows=-1), dict(activation=1), dict(activation=1, z_codes=F, z_scale=F),
                                dict(z_codes=F, z_scale=F), dict(dz=F), dict(dh=F), dict(dresidual=F), dict(eps=math.nan), dict(dy=ODD),
                                dict(h_codes=ODD), dict(dx=ODD), dict(ws=ODD), dict(dh=ODD, dresidual=F)])
def test_norm_gate_bwd8_refusals(lib, kw):
    assert _norm_b(lib, **kw) == gdn.GDN_EINVAL


def test_norm_gate_with_codes_widths_and_workspace(lib):
    for D in (4, 130, 16392):
        assert _norm(lib, D=D) == gdn.GDN_EUNSUPPORTED
        assert _norm_b(lib, D=D) == gdn.GDN_EUNSUPPORTED
    assert _norm_b(lib, bytes=8) == gdn.GDN_EWORKSPACE
    assert _norm_b(lib, ws=None) == gdn.GDN_EWORKSPACE
    assert _norm(lib, rows=0, x=None, y=None, h_codes=None, h_scale=None) == gdn.GDN_OK


def test_python_entries_refuse_the_cpu(lib):
    q = torch.zeros(4, 2, 64, dtype=BF)
    lse = torch.zeros(4, 2)
    codes, scale = torch.zeros(4, 128).to(torch.float8_e4m3fn), torch.ones(4, 1)
    x = torch.zeros(4, 128, dtype=BF)
    for call in (lambda: gdn.gdn_attention_fwd(q, q, q), lambda: gdn.gdn_attention_bwd(q, q, q, q, q, lse), lambda: gdn.gdn_act8_save(x),
                 lambda: gdn.gdn_act8_load(codes, scale), lambda: gdn.gdn_norm_gate_save8(x, torch.ones(128)),
                 lambda: gdn.gdn_norm_gate_bwd8(x, codes, scale, torch.ones(128))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        gdn.gdn_attention_fwd(None, q, q)
    with pytest.raises(ValueError, match="activation"):
        gdn.gdn_norm_gate_save8(x, torch.ones(128), z=x, activation="tanh")


@pytest.mark.parametrize("N", [1, 7, 100, 1024, 4096, 65535])
@pytest.mark.parametrize("T,Tk", [(10, 10), (37, 37), (300, 64), (64, 300), (4096, 1), (1, 9000)])
def test_attention_workspace_of_few_tokens(lib, N, T, Tk):
    """What empty sequences add is nothing: a row has 1024 bytes a head at most, and the walks of all keys' tiles (a tile
    has a key at least) are cut into 8 pieces each at most, and into twice the 152 SMs and one for each tile in all."""
    for HQ, HK, D in ((8, 2, 128), (1, 1, 64), (32, 32, 128)):
        pieces = min(8 * Tk * HK, 2 * 152 + min(Tk * HK, 2 * 152))
        assert 0 < gdn.attention_bwd_workspace_size(N, T, Tk, HQ, HK, D) <= 16 + 1024 * HQ * T + pieces * 2 * 128 * D * 4


@pytest.mark.parametrize("which", ["N", "Tq", "Tk", "HQ", "HK", "D"])
def test_attention_workspace_serves_smaller_calls(lib, which):
    """The workspace of one call is enough for every call of smaller sizes."""
    order = ("N", "Tq", "Tk", "HQ", "HK", "D")
    lengths = sorted({m for x in range(17) for m in (2 ** x - 1, 2 ** x, 2 ** x + 1, 5 << x)})
    ranges = dict(N=[n for n in lengths if 0 < n < 65536], Tq=lengths, Tk=lengths, HQ=range(8, 264, 8), HK=[1, 2, 4, 8], D=[64, 128])
    bases = [(1, 8192, 8192, 32, 4, 128), (24, 27160, 27160, 32, 4, 128), (1, 256, 256, 8, 2, 64), (300, 1000, 64, 8, 8, 128),
             (4096, 50, 16384, 64, 1, 64), (1, 1, 40000, 8, 1, 128)]
    for base in bases:
        sizes = dict(zip(order, base))
        got = [gdn.attention_bwd_workspace_size(*(x if n == which else sizes[n] for n in order)) for x in ranges[which]
               if which != "HK" or sizes["HQ"] % x == 0]
        assert all(a <= b for a, b in zip(got, got[1:])), (base, got)
        assert got[0] > 0


def test_attention_gradients_of_too_many_tiles(lib):
    """Tiles of all heads past 2^31: refused as not supported, with no size of a workspace, rather than by the launch."""
    big = dict(N=65535, cu=F, Tq=100000, Tk=100000, HQ=65535, HK=1, D=64, ldq=65535 * 64)
    assert gdn.attention_bwd_workspace_size(65535, 100000, 100000, 65535, 1, 64) == 0
    assert _bwd(lib, **big) == gdn.GDN_EUNSUPPORTED
    assert _bwd(lib, **dict(big, HK=65535, ldk=65535 * 64, ldv=65535 * 64)) == gdn.GDN_EUNSUPPORTED
    assert gdn.attention_bwd_workspace_size(65535, 32000, 32000, 65535, 1, 64) > 0
