"""Argument checks of the cache append and the attention calls (host only: every call here
fails validation, or is empty, before any kernel is launched)."""
import pytest
import torch

import draft_sampling_lossless_amd as dsl

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE, FAKE_ODD = 0x100000, 0x100004


def _err():
    return dsl.load().dspark_last_error().decode()


def _append(**kw):
    a = dict(q=FAKE, q_stride=1024, k=FAKE, k_stride=256, v=FAKE, v_stride=256, qnorm_w=FAKE, knorm_w=FAKE,
             positions=FAKE, slots=FAKE, q_out=FAKE, q_out_stride=1024, k_out=None, k_out_stride=0, k_cache=FAKE,
             v_cache=FAKE, M=4, nh=8, nkv=2, hd=128, num_slots=64, eps=1e-6, theta=1e6, stream=None)
    a.update(kw)
    return dsl.load().dspark_kv_append(*a.values())


def test_append_validation(dspark_lib):
    assert _append(M=0) == OK
    assert _append(M=-1) == INVALID
    assert _append(M=(1 << 22) + 1) == UNSUPPORTED
    assert _append(hd=96) == UNSUPPORTED and "hd" in _err()
    assert _append(hd=0) == INVALID and _append(hd=127) == INVALID
    assert _append(nkv=0) == INVALID and _append(nh=0) == INVALID
    assert _append(nh=1025, q_stride=1 << 20, q_out_stride=1 << 20) == UNSUPPORTED
    assert _append(num_slots=0) == INVALID
    assert _append(eps=-1.0) == INVALID and _append(eps=float("nan")) == INVALID
    assert _append(theta=0.0) == INVALID and _append(theta=float("inf")) == INVALID
    assert _append(q_out=None) == INVALID and "q_out" in _err()
    assert _append(q=None) == INVALID
    assert _append(q_stride=1016) == INVALID and _append(q_stride=1028) == INVALID
    assert _append(k_stride=255) == INVALID and _append(v_stride=0) == INVALID
    assert _append(k_out=FAKE, k_out_stride=128) == INVALID
    assert _append(k_out=FAKE, k_out_stride=512) == INVALID and "in place" in _err()
    assert _append(q_out_stride=2048) == INVALID and "in place" in _err()
    assert _append(k=None) == INVALID and _append(v=FAKE_ODD) == INVALID and "aligned" in _err()
    assert _append(q=FAKE_ODD) == INVALID and _append(knorm_w=FAKE_ODD) == INVALID
    assert _append(positions=None) == INVALID and _append(slots=None) == INVALID
    assert _append(k_cache=None) == INVALID and _append(v_cache=FAKE_ODD) == INVALID


def _paged(**kw):
    a = dict(q=FAKE, q_stride=1024, k_cache=FAKE, v_cache=FAKE, page_table=FAKE, kv_len=FAKE, cu_q=FAKE, out=FAKE,
             lse=None, T=4, B=2, max_q=3, nh=8, nkv=2, hd=128, page_size=16, max_pages=8, num_pages=32, causal=1,
             scale=0.1, workspace=FAKE, workspace_bytes=1 << 30, stream=None)
    a.update(kw)
    return dsl.load().dspark_paged_attention(*a.values())


def test_paged_validation(dspark_lib):
    assert _paged(T=0) == OK
    assert _paged(T=-1) == INVALID and _paged(B=0) == INVALID and _paged(B=4097) == UNSUPPORTED
    assert _paged(nh=9) == INVALID and _paged(nkv=0) == INVALID and _paged(nkv=3) == INVALID
    assert _paged(nh=2048, q_stride=1 << 20) == UNSUPPORTED
    assert _paged(hd=96) == UNSUPPORTED and _paged(hd=32) == UNSUPPORTED and _paged(hd=-2) == INVALID
    assert _paged(T=1 << 28) == UNSUPPORTED and "2^30" in _err()
    assert _paged(scale=0.0) == INVALID and _paged(scale=float("nan")) == INVALID and _paged(scale=-1.0) == INVALID
    assert _paged(q_stride=1000) == INVALID and _paged(q_stride=1028) == INVALID
    assert _paged(max_q=0) == INVALID and _paged(max_q=129) == UNSUPPORTED
    assert _paged(page_size=0) == INVALID and _paged(page_size=24) == UNSUPPORTED
    assert _paged(max_pages=0) == INVALID and _paged(num_pages=0) == INVALID
    assert _paged(num_pages=1 << 27) == UNSUPPORTED and _paged(max_pages=1 << 27) == UNSUPPORTED
    assert _paged(max_pages=(1 << 26) + 1) == UNSUPPORTED                # more than 2^30 keys of a request
    assert _paged(causal=2) == INVALID
    for name in ("q", "k_cache", "v_cache", "page_table", "kv_len", "cu_q", "out"):
        assert _paged(**{name: None}) == INVALID and name in _err()
    for name in ("q", "k_cache", "v_cache", "out", "workspace"):
        assert _paged(**{name: FAKE_ODD}) == INVALID and "aligned" in _err()
    assert _paged(workspace=None) == WORKSPACE
    need = dsl.paged_attention_workspace_size(4, 2, 3, 8, 2, 128)
    assert need > 0 and _paged(workspace_bytes=need - 1) == WORKSPACE and "too small" in _err()
    assert dsl.paged_attention_workspace_size(0, 2, 3, 8, 2, 128) == 0
    assert dsl.paged_attention_workspace_size(4352, 256, 17, 32, 8, 128) < 512 << 20


def _prompt(**kw):
    a = dict(q=FAKE, q_stride=1024, k=FAKE, k_stride=256, v=FAKE, v_stride=256, cu_seqlens=FAKE, out=FAKE, lse=None,
             T=4, B=2, nh=8, nkv=2, hd=128, causal=1, scale=0.1, stream=None)
    a.update(kw)
    return dsl.load().dspark_prompt_attention(*a.values())


def test_prompt_validation(dspark_lib):
    assert _prompt(T=0) == OK
    assert _prompt(T=-4) == INVALID and _prompt(B=0) == INVALID and _prompt(B=4097) == UNSUPPORTED
    assert _prompt(hd=80) == UNSUPPORTED and _prompt(nh=7) == INVALID
    assert _prompt(q_stride=512) == INVALID and _prompt(k_stride=260) == INVALID and _prompt(v_stride=128) == INVALID
    assert _prompt(k_stride=1 << 24) == UNSUPPORTED and _prompt(v_stride=1 << 30) == UNSUPPORTED
    assert _prompt(causal=-1) == INVALID and _prompt(scale=float("inf")) == INVALID
    for name in ("q", "k", "v", "cu_seqlens", "out"):
        assert _prompt(**{name: None}) == INVALID and name in _err()
    for name in ("q", "k", "v", "out"):
        assert _prompt(**{name: FAKE_ODD}) == INVALID and "aligned" in _err()


@pytest.mark.parametrize("call", [_paged, _prompt])
def test_scales_whose_factor_is_no_float_are_refused(dspark_lib, call):
    for scale in (2.0 ** 126.1, 2.0 ** 127, 2.5e38, 3.4e38):
        assert call(scale=scale) == UNSUPPORTED and "2^126" in _err()
    assert call(scale=2.0 ** 126, T=0) == OK and call(scale=1e-45, T=0) == OK


def test_binding_refuses_host_tensors_and_wrong_types(dspark_lib):
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        dsl.kv_append(x, x, i, i.long(), x, x)
    with pytest.raises(ValueError):
        dsl.paged_attention(x, x, x, i[None], i, i, 1, 1)
    with pytest.raises(ValueError):
        dsl.prompt_attention(x, x, x, i)
    with pytest.raises(TypeError):
        dsl.prompt_attention(None, x, x, i)
