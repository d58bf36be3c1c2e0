"""Refusals of the decode step's operators (append with rotation, attention over a
shared prefix, token sampling) without a GPU: the library's host checks (fake
device addresses, no CUDA call on these paths) and the binding's checks of tensors."""

import ctypes
import random
import subprocess

import pytest
import torch

from speculative_decoding_tree_sv_gb300 import binding as sv
from speculative_decoding_tree_sv_gb300 import build

A = 1 << 20  # a 16-byte aligned address that is never used
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return sv.load()


def filled(p, kw):
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def rope(**over):
    return filled(sv.sv_rope_params(), {**dict(
        batch=2, num_q_heads=32, num_kv_heads=8, head_dim=128, rotary_dim=128, page_size=16, num_pages=100, total_tokens=40,
        max_pages_per_seq=20, dtype=0, interleaved=0, flags=0, amplitude=0.0, q_stride=0, q_out_stride=0, kv_stride=0, q=A,
        k=A, v=A, q_out=2 * A, k_cache=A, v_cache=A, block_table=A, ctx_lens=A, cu_tokens=A, positions=None, inv_freq=A,
        new_ctx_lens=None, workspace=None, workspace_bytes=0), **over})


@pytest.mark.parametrize("over,status", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(q_out=None), 1), (dict(k_cache=None), 1),
    (dict(v_cache=None), 1), (dict(block_table=None), 1), (dict(ctx_lens=None), 1), (dict(cu_tokens=None), 1),
    (dict(inv_freq=None), 1), (dict(q=A + 8), 1), (dict(k=A + 2), 1), (dict(v=A + 4), 1), (dict(q_out=A + 8), 1),
    (dict(k_cache=A + 8), 1), (dict(v_cache=A + 8), 1), (dict(inv_freq=A + 2), 1), (dict(positions=A + 1), 1),
    (dict(batch=0), 1), (dict(num_q_heads=-1), 1), (dict(num_kv_heads=0), 1), (dict(num_pages=0), 1),
    (dict(max_pages_per_seq=0), 1), (dict(page_size=0), 1), (dict(total_tokens=-1), 1), (dict(flags=1), 1),
    (dict(total_tokens=(1 << 30) + 1), 2), (dict(num_q_heads=65536), 2), (dict(num_kv_heads=65536), 2),
    (dict(dtype=2), 2), (dict(dtype=-1), 2), (dict(head_dim=120), 2), (dict(head_dim=272), 2), (dict(head_dim=0), 2),
    (dict(rotary_dim=0), 1), (dict(rotary_dim=144), 1), (dict(rotary_dim=24), 2), (dict(rotary_dim=-16), 1),
    (dict(amplitude=NAN), 1), (dict(amplitude=INF), 1), (dict(q_stride=4088), 1), (dict(q_stride=4100), 1),
    (dict(q_out_stride=4088), 1), (dict(kv_stride=1016), 1), (dict(kv_stride=1028), 1), (dict(kv_stride=1 << 39), 1),
    (dict(q_out=A, q_stride=4104), 1),               # in place wants one stride
    (dict(new_ctx_lens=A), 1),                       # the context lengths themselves
    (dict(workspace=A, workspace_bytes=255), 4), (dict(workspace=A + 2, workspace_bytes=256), 1),
])
def test_rope_append_refuses(lib, over, status):
    assert lib.sv_rope_append(ctypes.byref(rope(**over)), None) == status


def prefix(**over):
    return filled(sv.sv_prefix_params(), {**dict(
        batch=4, num_q_heads=32, num_kv_heads=8, head_dim=128, page_size=16, num_pages=100, total_tokens=40, max_tokens=39,
        max_pages_per_seq=20, dtype=0, num_groups=2, max_group_tokens=40, sm_scale=0.0, flags=0, q_stride=0, out_stride=0,
        q=A, k_cache=A, v_cache=A, block_table=A, ctx_lens=A, cu_tokens=A, cu_groups=A, prefix_lens=A, out=A, lse=None,
        workspace=A, workspace_bytes=1 << 40), **over})


@pytest.mark.parametrize("over,status", [
    (dict(q=None), 1), (dict(k_cache=None), 1), (dict(v_cache=None), 1), (dict(block_table=None), 1),
    (dict(ctx_lens=None), 1), (dict(cu_tokens=None), 1), (dict(cu_groups=None), 1), (dict(prefix_lens=None), 1),
    (dict(out=None), 1), (dict(q=A + 8), 1), (dict(k_cache=A + 2), 1), (dict(out=A + 4), 1), (dict(workspace=A + 8), 1),
    (dict(batch=0), 1), (dict(batch=65536), 2), (dict(num_groups=0), 1), (dict(num_groups=5), 1),
    (dict(max_group_tokens=-1), 1), (dict(num_kv_heads=0), 1), (dict(num_q_heads=30), 1),
    (dict(num_q_heads=129, num_kv_heads=1), 2), (dict(head_dim=96), 2), (dict(page_size=32), 2), (dict(num_pages=0), 1),
    (dict(max_pages_per_seq=0), 1), (dict(max_pages_per_seq=1 << 27), 2), (dict(total_tokens=-1), 1),
    (dict(total_tokens=(1 << 30) + 1), 2), (dict(total_tokens=1 << 30, num_q_heads=128), 2), (dict(max_tokens=-1), 1),
    (dict(dtype=2), 2), (dict(flags=1), 1), (dict(sm_scale=NAN), 1), (dict(q_stride=4095), 1), (dict(q_stride=4100), 1),
    (dict(out_stride=4088), 1), (dict(workspace=None), 4), (dict(workspace_bytes=300), 4),
    (dict(batch=65535, num_kv_heads=16384, num_q_heads=16384), 2),
])
def test_prefix_attention_refuses(lib, over, status):
    assert lib.sv_prefix_attention(ctypes.byref(prefix(**over)), None) == status


def sample(**over):
    return filled(sv.sv_sample_params(), {**dict(
        rows=4, vocab=1000, dtype=2, flags=0, logits_stride=0, probs_stride=0, logits=A, uniforms=A, temperature=None,
        top_k=None, top_p=None, min_p=None, tokens=A, logprobs=None, probs=None, workspace=None, workspace_bytes=0), **over})


@pytest.mark.parametrize("over,status", [
    (dict(logits=None), 1), (dict(uniforms=None), 1), (dict(tokens=None), 1), (dict(rows=-1), 1), (dict(vocab=0), 1),
    (dict(vocab=(1 << 18) + 1), 2), (dict(rows=(1 << 24) + 1), 2), (dict(dtype=3), 2), (dict(dtype=-1), 2), (dict(flags=1), 1),
    (dict(logits_stride=999), 1), (dict(probs_stride=999), 1), (dict(logits_stride=-1000), 1),
    (dict(logits_stride=(1 << 38) + 1), 1), (dict(logits=A + 2), 1), (dict(dtype=0, logits=A + 1), 1),
    (dict(uniforms=A + 2), 1), (dict(temperature=A + 2), 1), (dict(top_k=A + 1), 1), (dict(top_p=A + 2), 1),
    (dict(min_p=A + 3), 1), (dict(tokens=A + 2), 1), (dict(logprobs=A + 2), 1), (dict(probs=A + 2), 1),
    (dict(probs=A), 1),                              # in place
    (dict(workspace=A + 2, workspace_bytes=256), 1), (dict(workspace=A, workspace_bytes=255), 4),
])
def test_sample_tokens_refuses(lib, over, status):
    assert lib.sv_sample_tokens(ctypes.byref(sample(**over)), None) == status


def test_nothing_to_do_and_null(lib):
    n = ctypes.c_size_t(0)
    assert lib.sv_rope_append(None, None) == 1 and lib.sv_sample_tokens(None, None) == 1
    assert lib.sv_prefix_attention(None, None) == 1
    assert lib.sv_prefix_attention_workspace_size(None, ctypes.byref(n)) == 1
    assert lib.sv_prefix_attention_workspace_size(ctypes.byref(prefix()), None) == 1
    for over in (dict(total_tokens=0), dict(max_tokens=0), dict(max_group_tokens=0), dict(total_tokens=0, q=None, out=None)):
        assert lib.sv_prefix_attention(ctypes.byref(prefix(**over)), None) == 0
    assert lib.sv_sample_tokens(ctypes.byref(sample(rows=0)), None) == 0
    assert lib.sv_sample_tokens(ctypes.byref(sample(rows=0, logits=None, uniforms=None, tokens=None)), None) == 0
    if not torch.cuda.is_available():  # (the append launches, for the lengths; 3: no device to launch on)
        assert lib.sv_rope_append(ctypes.byref(rope(total_tokens=0, q=None, k=None, v=None, q_out=None)), None) == 3
        assert lib.sv_rope_append(ctypes.byref(rope(num_q_heads=0, q=None, q_out=None)), None) == 3


def test_prefix_workspace_holds_the_partials(lib):
    size = sv.sv_prefix_attention_workspace_size
    row = 32 * (128 + 1) * 4                      # a token's fp32 rows and log sums, all heads
    assert size(prefix()) >= 2 * 40 * row         # of the prefix and of its own keys
    # a group is shared up to an M tile of rows (32 tokens here) per sequence: no more rows lie there
    assert size(prefix(total_tokens=4000, max_tokens=1000, max_group_tokens=2000)) >= 2 * 4 * 32 * row
    assert size(prefix(total_tokens=0)) >= 256
    # a group may be as large as the call: the bound of its tokens beyond that changes nothing
    assert size(prefix(max_group_tokens=1 << 30)) == size(prefix(max_group_tokens=40))


def i(*s):
    return torch.zeros(s, dtype=torch.int32)


def h(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def rope_tensors():
    return dict(q=h(5, 8, 64), k=h(5, 2, 64), v=h(5, 2, 64), q_out=h(5, 8, 64), k_cache=h(6, 2, 16, 64),
                v_cache=h(6, 2, 16, 64), block_table=i(2, 3), ctx_lens=i(2), cu_tokens=i(3), inv_freq=torch.zeros(32))


def test_binding_of_the_append_refuses(lib):
    good = rope_tensors()
    with pytest.raises(ValueError, match="device memory"):
        sv.sv_rope_append(**good)
    rows = torch.zeros(6 * 512, dtype=torch.bfloat16)
    for bad, text in (
            (dict(q=h(5, 8, 64).half()), "cache's type"), (dict(q=None), "come together"), (dict(q_out=None), "come together"),
            (dict(q=h(4, 8, 64)), "q must be"), (dict(q_out=h(5, 4, 64)), "q_out must be"), (dict(v=h(5, 4, 64)), "v must be"),
            (dict(k=h(5, 128)), "k must be"), (dict(k=h(5, 2, 32), v=h(5, 2, 32)), "k must be"),
            (dict(v=h(5, 64, 2).transpose(1, 2)), "heads of v"), (dict(v=h(5, 3, 64)[:, :2]), "same strides"),
            (dict(q=rows.as_strided((5, 8, 64), (0, 64, 1))), "rows of q overlap"),
            (dict(q_out=rows.as_strided((5, 8, 64), (504, 64, 1))), "rows of q_out overlap"),
            (dict(k=rows.as_strided((5, 2, 64), (64, 64, 1))), "rows of k overlap"),
            (dict(v_cache=h(6, 2, 16, 32)), "same shape"), (dict(k_cache=h(2, 6, 2, 16, 64), v_cache=h(2, 6, 2, 16, 64)), "one layer"),
            (dict(block_table=i(6)), r"\[batch, max_pages\]"), (dict(block_table=torch.zeros(2, 3)), "int32"),
            (dict(ctx_lens=i(3)), "2 elements"), (dict(cu_tokens=i(2)), "3 elements"), (dict(inv_freq=torch.zeros(2, 16)), "inv_freq"),
            (dict(inv_freq=torch.zeros(32, dtype=torch.float64)), "inv_freq"), (dict(inv_freq=torch.zeros(64)[::2]), "inv_freq"),
            (dict(positions=i(4)), "5 elements"), (dict(positions=torch.zeros(5, dtype=torch.int64)), "int32"),
            (dict(new_ctx_lens=i(3)), "2 elements")):
        with pytest.raises(ValueError, match=text):
            sv.sv_rope_append(**{**good, **bad})


def prefix_tensors():
    return dict(q=h(5, 8, 64), k_cache=h(6, 2, 16, 64), v_cache=h(6, 2, 16, 64), block_table=i(2, 3), ctx_lens=i(2),
                cu_tokens=i(3), cu_groups=i(2), prefix_lens=i(1), out=h(5, 8, 64), max_tokens=4, max_group_tokens=5)


def test_binding_of_the_prefix_attention_refuses():
    good = prefix_tensors()
    with pytest.raises(ValueError, match="device memory"):
        sv.make_prefix_params(**good)
    for bad, text in ((dict(cu_groups=i(1)), "cu_groups"), (dict(cu_groups=torch.zeros(2)), "int32"),
                      (dict(prefix_lens=i(2)), "1 elements"), (dict(prefix_lens=torch.zeros(1)), "int32"),
                      (dict(q=h(5, 8, 64).float()), "bfloat16 or float16"), (dict(out=h(5, 8, 32)), "must both be"),
                      (dict(k_cache=h(6, 2, 16, 128), v_cache=h(6, 2, 16, 128)), "head_dim"), (dict(ctx_lens=i(3)), "2 elements"),
                      (dict(lse=torch.zeros(5, 4)), "lse"), (dict(q=h(5, 64, 8).transpose(1, 2)), "heads of q"),
                      (dict(max_group_tokens=1 << 31), "max_group_tokens does not fit"),
                      (dict(max_tokens=(1 << 32) + 5), "max_tokens does not fit")):
        with pytest.raises(ValueError, match=text):
            sv.make_prefix_params(**{**good, **bad})


def test_binding_of_the_sampling_refuses(lib):
    f = lambda *s: torch.zeros(s)  # noqa: E731
    good = dict(logits=f(3, 10), uniforms=f(3), tokens=i(3))
    with pytest.raises(ValueError, match="device memory"):
        sv.sv_sample_tokens(**good)
    for bad, text in ((dict(logits=f(3, 10).double()), "float32, bfloat16 or float16"), (dict(logits=f(30)), "logits must be"),
                      (dict(logits=f(10, 3).t()), "rows of logits must be contiguous"),
                      (dict(logits=f(1, 10).expand(3, 10)), "rows of logits overlap"), (dict(uniforms=None), "uniforms"),
                      (dict(uniforms=f(2)), "uniforms"), (dict(uniforms=f(3).double()), "uniforms"), (dict(tokens=i(2)), "3 elements"),
                      (dict(tokens=torch.zeros(3, dtype=torch.int64)), "int32"), (dict(temperature=f(1)), "temperature"),
                      (dict(top_k=f(3)), "int32"), (dict(top_p=f(6)[::2]), "top_p"), (dict(min_p=f(4)), "min_p"),
                      (dict(logprobs=f(3).half()), "logprobs"), (dict(probs=f(3, 9)), "probs must be"),
                      (dict(probs=f(3, 10).half()), "probs must be float32"), (dict(probs=f(1, 10).expand(3, 10)), "rows of probs overlap")):
        with pytest.raises(ValueError, match=text):
            sv.sv_sample_tokens(**{**good, **bad})


def test_the_append_with_rotation_signals_nothing_early():
    """As the other kernels that write tables, lengths or context pages: a tree
    attention with SV_ATTN_EARLY_CONTEXT reads them at the signal."""
    with open(f"{build.CSRC}/rope_append.cu") as f:
        source = f.read()
    assert "griddep_wait();" in source and "launch_dependents" not in source


KERNELS = r"""
#include "prefix_kernels.h"
extern "C" int kernels(long long total, long long batch, long long most, long long group, long long heads) {
  const sv::PrefixKernels k = sv::prefix_kernels(total, batch, most, group, heads, 16);
  return (k.rows ? 1 : 0) | (k.tiles ? 2 : 0);
}
"""


def test_every_entry_of_a_prefix_call_has_a_kernel(tmp_path):
    """Whatever the token rows behind the last sequence and the host's bounds: an entry of n tokens goes to the row kernel
    up to 16 rows per KV head where that is in the call, else to the tile kernel, which then is."""
    source, module = tmp_path / "kernels.cpp", tmp_path / "kernels.so"
    source.write_text(KERNELS)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", build.CSRC, "-o", module, source], check=True)
    kernels = ctypes.CDLL(str(module)).kernels
    kernels.argtypes = [ctypes.c_longlong] * 5
    rng = random.Random(1)
    for lens in [[1], [1] * 4, [1] * 64, [0, 1], [2, 9], [5, 1, 1], [17], [40, 30]] + [
            [rng.randint(0, 30) for _ in range(rng.randint(1, 12))] for _ in range(60)]:
        for heads in (1, 2, 4, 5, 8, 16, 17, 32, 128):
            for padding in (0, 1, 2, 3, 4, 7, 8, 40, 900, 1 << 29):
                for loose in (0, 1, 50):
                    for group in (max(lens), sum(lens)):
                        taken = kernels(sum(lens) + padding, len(lens), max(1, max(lens)) + loose, max(1, group) + loose, heads)
                        for n in lens + [group]:
                            by_rows = taken & 1 and n * heads <= 16
                            assert n == 0 or by_rows or taken & 2, (lens, heads, padding, loose, group)
    # a padded step of single tokens stays in the row kernel
    assert kernels(128, 64, 1, 4, 4) == 1 and kernels(128, 64, 1, 64, 4) == 3
