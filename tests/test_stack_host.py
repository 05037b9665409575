"""Host-side checks of the operators around the recurrence: the C entries refuse bad arguments before any CUDA work,
the Python entries refuse wrong types, devices and layouts, and the rotary frequencies follow their formulas.  Runs
without a GPU."""
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


def _call(lib, name, order, **kw):
    return getattr(lib, name)(*[kw[k] for k in order.split()])


NORM = "x residual z weight res_scale eps activation rows D z_rows z_stride y h stream"


def _norm(lib, **kw):
    a = dict(x=F, residual=None, z=None, weight=F, res_scale=1.0, eps=1e-6, activation=0, rows=4, D=128, z_rows=0, z_stride=0,
             y=F, h=None, stream=None)
    a.update(kw)
    return _call(lib, "gdn_norm_gate", NORM, **a)


@pytest.mark.parametrize("kw", [dict(x=None), dict(weight=None), dict(y=None), dict(D=0), dict(rows=-1), dict(activation=3, z=F),
                                dict(activation=-1), dict(activation=1), dict(z=F), dict(residual=F), dict(h=F), dict(eps=-1.0),
                                dict(eps=math.nan), dict(activation=1, z=F, z_rows=-1)])
def test_norm_gate_refusals(lib, kw):
    assert _norm(lib, **kw) == gdn.GDN_EINVAL


def test_norm_gate_without_rows(lib):
    assert _norm(lib, rows=0, x=None, weight=None, y=None) == gdn.GDN_OK


@pytest.mark.parametrize("kw", [dict(activation=1), dict(activation=2, residual=None, h=None), dict(residual=F), dict(h=F)])
def test_norm_gate_of_an_empty_batch(lib, kw):
    """Empty tensors have null pointers: a call without rows does nothing, whatever it would do with some."""
    assert _norm(lib, rows=0, x=None, y=None, **kw) == gdn.GDN_OK


NORM_B = ("dy h z dh weight res_scale eps activation rows D z_rows z_stride dx dresidual dz dweight workspace workspace_bytes "
          "stream")


def _norm_b(lib, **kw):
    a = dict(dy=F, h=F, z=None, dh=None, weight=F, res_scale=1.0, eps=1e-6, activation=0, rows=4, D=128, z_rows=0, z_stride=0,
             dx=F, dresidual=None, dz=None, dweight=F, workspace=F, workspace_bytes=1 << 40, stream=None)
    a.update(kw)
    return _call(lib, "gdn_norm_gate_bwd", NORM_B, **a)


@pytest.mark.parametrize("kw", [dict(dy=None), dict(h=None), dict(weight=None), dict(dx=None), dict(dweight=None), dict(D=-1),
                                dict(rows=-1), dict(activation=1, dz=F), dict(activation=1, z=F), dict(z=F), dict(dz=F),
                                dict(dh=F), dict(dresidual=F), dict(eps=math.nan), dict(workspace=ODD)])
def test_norm_gate_bwd_refusals(lib, kw):
    assert _norm_b(lib, **kw) == gdn.GDN_EINVAL


def test_norm_gate_bwd_workspace(lib):
    need = lib.gdn_norm_gate_bwd_workspace_size(4, 128)
    assert need > 0 and lib.gdn_norm_gate_bwd_workspace_size(-1, 128) == 0 and lib.gdn_norm_gate_bwd_workspace_size(4, 0) == 0
    assert _norm_b(lib, workspace_bytes=need - 1) == gdn.GDN_EWORKSPACE
    assert _norm_b(lib, workspace=None) == gdn.GDN_EWORKSPACE


ROPE = ("q k positions inv_freq T HQ HK D rotary_dim interleaved inverse attention_factor ldq ldk q_out k_out stream")


def _rope(lib, **kw):
    a = dict(q=F, k=F, positions=F, inv_freq=F, T=4, HQ=4, HK=2, D=64, rotary_dim=32, interleaved=0, inverse=0,
             attention_factor=1.0, ldq=256, ldk=128, q_out=ODD, k_out=ODD, stream=None)
    a.update(kw)
    return _call(lib, "gdn_rope", ROPE, **a)


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(positions=None), dict(inv_freq=None), dict(q_out=None),
                                dict(k_out=None), dict(T=-1), dict(HQ=0), dict(HK=-1), dict(D=0), dict(rotary_dim=0),
                                dict(rotary_dim=31), dict(rotary_dim=66), dict(ldq=255), dict(ldk=127),
                                dict(q_out=F, ldq=264), dict(k_out=F, ldk=136)])
def test_rope_refusals(lib, kw):
    assert _rope(lib, **kw) == gdn.GDN_EINVAL


def test_rope_limits(lib):
    assert _rope(lib, D=8194, rotary_dim=8194, ldq=4 * 8194, ldk=2 * 8194) == gdn.GDN_EUNSUPPORTED
    assert _rope(lib, T=0, q=None, q_out=None) == gdn.GDN_OK


PLAN = ("cached_lens cu_seqlens N T block_table width free_pages F num_free page_size seq_lens slot_mapping positions "
        "num_free_out dev_status stream")


@pytest.mark.parametrize("kw", [dict(cached_lens=None), dict(cu_seqlens=None), dict(N=-1), dict(T=-1), dict(block_table=None),
                                dict(width=-1), dict(free_pages=None), dict(F=-1), dict(num_free=None), dict(page_size=0),
                                dict(seq_lens=None), dict(slot_mapping=None), dict(positions=None), dict(num_free_out=None),
                                dict(num_free_out=F)])
def test_paged_plan_refusals(lib, kw):
    a = dict(cached_lens=F, cu_seqlens=F, N=2, T=4, block_table=F, width=3, free_pages=F, F=5, num_free=F, page_size=16,
             seq_lens=F, slot_mapping=F, positions=F, num_free_out=ODD, dev_status=None, stream=None)
    a.update(kw)
    assert _call(lib, "gdn_paged_plan", PLAN, **a) == gdn.GDN_EINVAL


APPEND = "k v ldk ldv k_cache v_cache k_scale v_scale slot_mapping T P HK D page_size dev_status stream"


def _append(lib, **kw):
    a = dict(k=F, v=F, ldk=256, ldv=256, k_cache=F, v_cache=F, k_scale=F, v_scale=F, slot_mapping=F, T=3, P=4, HK=2, D=128,
             page_size=64, dev_status=None, stream=None)
    a.update(kw)
    return _call(lib, "gdn_kv8_append", APPEND, **a)


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(k_cache=None), dict(v_cache=None), dict(k_scale=None),
                                dict(v_scale=None), dict(slot_mapping=None), dict(T=-1), dict(P=0), dict(HK=0), dict(D=0),
                                dict(page_size=0), dict(ldk=255), dict(ldv=255), dict(P=1 << 26)])
def test_kv8_append_refusals(lib, kw):
    assert _append(lib, **kw) == gdn.GDN_EINVAL


def test_kv8_append_limits(lib):
    assert _append(lib, HK=32768, ldk=1 << 30, ldv=1 << 30) == gdn.GDN_EUNSUPPORTED
    assert _append(lib, T=0, k=None, v=None) == gdn.GDN_OK


def test_kv8_append_page_past_32_bits(lib):
    """A page's values of one head are counted in 32 bits (nothing is launched: the call is refused)."""
    assert _append(lib, P=1, HK=1, page_size=1 << 20, D=4096, ldk=4096, ldv=4096) == gdn.GDN_EUNSUPPORTED


ATTN = ("q ldq k_cache v_cache k_scale v_scale block_table width seq_lens cu_seqlens N T P HQ HK D page_size max_q_len "
        "max_seq_len scale o lse workspace workspace_bytes dev_status stream")


def _attn(lib, **kw):
    a = dict(q=F, ldq=512, k_cache=F, v_cache=F, k_scale=F, v_scale=F, block_table=F, width=4, seq_lens=F, cu_seqlens=F, N=2,
             T=6, P=9, HQ=4, HK=2, D=128, page_size=64, max_q_len=4, max_seq_len=256, scale=-1.0, o=F, lse=None, workspace=F,
             workspace_bytes=1 << 40, dev_status=None, stream=None)
    a.update(kw)
    return _call(lib, "gdn_kv8_attention", ATTN, **a)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(k_cache=None), dict(v_cache=None), dict(k_scale=None), dict(v_scale=None), dict(block_table=None),
    dict(seq_lens=None), dict(o=None), dict(N=-1), dict(T=-1), dict(P=-1), dict(P=0), dict(HQ=0), dict(HK=0), dict(HQ=5),
    dict(width=-1), dict(page_size=0), dict(D=0), dict(max_q_len=0), dict(max_q_len=-1), dict(max_seq_len=-1), dict(max_seq_len=257),
    dict(cu_seqlens=None), dict(ldq=511), dict(ldq=516), dict(q=ODD), dict(k_cache=ODD), dict(v_cache=ODD), dict(o=ODD),
    dict(workspace=ODD)])
def test_kv8_attention_refusals(lib, kw):
    assert _attn(lib, **kw) == gdn.GDN_EINVAL


@pytest.mark.parametrize("kw", [dict(D=96, ldq=384), dict(D=256, ldq=1024), dict(page_size=8, max_seq_len=32),
                                dict(page_size=256), dict(N=65536), dict(HQ=65536, HK=65536, ldq=65536 * 128), dict(P=1 << 30)])
def test_kv8_attention_limits(lib, kw):
    assert _attn(lib, **kw) == gdn.GDN_EUNSUPPORTED


def test_kv8_attention_workspace(lib):
    size = gdn.kv8_attention_workspace_size
    for new in (1, 4, 40, 4000):  # few tokens, some, many: no more than 64 MB, and refused when short of a byte
        need = size(2, 2 * new, 4, 2, 128, new, 256)
        assert 0 < need < 1 << 26
        assert _attn(lib, T=2 * new, max_q_len=new, workspace_bytes=need - 1) == gdn.GDN_EWORKSPACE
        assert _attn(lib, T=2 * new, max_q_len=new, workspace=None) == gdn.GDN_EWORKSPACE
    assert size(0, 0, 4, 2, 128, 1, 256) == 0 and size(2, 2, 4, 2, 96, 1, 256) == 0
    assert _attn(lib, N=0, T=0, q=None, o=None) == gdn.GDN_OK


# ------------------------------------------------------------ Python entries
def _i(*v):
    return torch.tensor(v, dtype=torch.int32)


def _cache(P=4, H=2, bs=16, D=64):
    z = torch.zeros(P, H, bs, D, dtype=torch.float8_e4m3fn)
    return [z, z.clone(), torch.ones(P, H), torch.ones(P, H)]


def test_python_entries_refuse_what_is_not_on_a_gpu(lib):
    x = torch.zeros(3, 2, 64, dtype=BF)
    with pytest.raises(ValueError):
        gdn.gdn_norm_gate(x, torch.ones(64))
    with pytest.raises(ValueError):
        gdn.gdn_norm_gate_bwd(x, x, torch.ones(64))
    with pytest.raises(ValueError):
        gdn.gdn_rope(x, x, _i(0, 1, 2), torch.ones(32))
    with pytest.raises(ValueError):
        gdn.gdn_paged_plan(_i(0), _i(0, 1), _i(0).view(1, 1), _i(0), _i(1), 16, 1)
    with pytest.raises(ValueError):
        gdn.gdn_kv8_append(x, x, *_cache(), _i(0, 1, 2))
    with pytest.raises(ValueError):
        gdn.gdn_kv8_attention(x, *_cache(), _i(0, 1, 2).view(3, 1), _i(1, 1, 1))


def test_python_entries_refuse_what_is_no_tensor_and_unknown_names(lib):
    x = torch.zeros(3, 2, 64, dtype=BF)
    with pytest.raises(TypeError):
        gdn.gdn_norm_gate([1.0], torch.ones(64))
    with pytest.raises(TypeError):
        gdn.gdn_rope(x, 3, _i(0, 1, 2), torch.ones(32))
    with pytest.raises(ValueError):
        gdn.gdn_norm_gate(x, torch.ones(64), activation="relu")
    with pytest.raises(ValueError):
        gdn.gdn_norm_gate_bwd(x, x, torch.ones(64), activation=7)


@pytest.mark.parametrize("stamp", ["another interpreter and PyTorch", None])
def test_binding_built_for_another_pytorch_is_refused(lib, tmp_path, monkeypatch, stamp):
    from gated_deltanet_chunked_chunk_gb300 import stack
    assert stack._load() is not None
    if stamp is not None:
        (tmp_path / "for").write_text(stamp)
    monkeypatch.setattr(gbuild, "STAMP", str(tmp_path / "for"))
    assert not gbuild.up_to_date()
    monkeypatch.setattr(stack, "_c", None)
    with pytest.raises(RuntimeError, match="build it again"):
        gdn.gdn_norm_gate(torch.zeros(3, 64, dtype=BF), torch.ones(64))


# --------------------------------------------------------- rotary frequencies
def test_rope_frequencies_formulas():
    inv, att = gdn.rope_frequencies(128, 10000.0)
    ref = torch.tensor([10000.0 ** (-2 * i / 128) for i in range(64)], dtype=torch.float64)
    assert inv.dtype == torch.float32 and att == 1.0 and torch.equal(inv, ref.float())
    lin, att = gdn.rope_frequencies(128, scaling="linear", factor=4.0)
    assert att == 1.0 and torch.equal(lin, (ref / 4).float())
    ntk, att = gdn.rope_frequencies(128, scaling="ntk", factor=8.0)
    assert att == 1.0 and ntk[0] == 1.0 and abs(float(ntk[-1]) / float(ref[-1] / 8) - 1) < 1e-6  # fastest stays, slowest / factor
    yarn, att = gdn.rope_frequencies(128, scaling="yarn", factor=16.0, original_max_position=4096)
    assert abs(att - (0.1 * math.log(16.0) + 1.0)) < 1e-12
    turns = 4096 * ref / (2 * math.pi)
    assert torch.equal(yarn[turns > 40], ref[turns > 40].float())                  # fast pairs as they were
    assert torch.allclose(yarn[turns < 0.8], (ref[turns < 0.8] / 16).float())      # slow ones by the factor
    assert (yarn <= ref.float()).all() and (yarn >= (ref / 16).float() * (1 - 1e-6)).all()
    same, _ = gdn.rope_frequencies(128, scaling="yarn", factor=1.0)
    assert torch.allclose(same, ref.float())
    assert gdn.rope_frequencies(2)[0].tolist() == [1.0]


@pytest.mark.parametrize("kw", [dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=8, base=0.0), dict(rotary_dim=8, base=math.inf),
                                dict(rotary_dim=8, scaling="linear", factor=0.5), dict(rotary_dim=8, scaling="other")])
def test_rope_frequencies_refusals(kw):
    with pytest.raises(ValueError):
        gdn.rope_frequencies(**kw)
