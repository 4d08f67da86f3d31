"""Host-only checks of the paged calls' Python arguments: what is no tensor, or a tensor of other
dimensions, is named in the error; numbers that the C ABI's 32 bits do not hold are refused instead of
wrapped; and the module does without PyTorch's private names."""
import os
import subprocess
import sys

import pytest
import torch

import prefill_only_cascade_gb300 as q

BF, I32 = torch.bfloat16, torch.int32


def cpu(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


DESC = q.make_paged_desc(2, 30, 8, 16, 2, 4, 2, 64)
PAGES = cpu(8, 16, 2, 64, dtype=BF)
APPEND = dict(k_new=cpu(2, 2, 64, dtype=BF), v_new=cpu(2, 2, 64, dtype=BF), start_pos=cpu(2, dtype=I32),
              block_table=cpu(2, 2, dtype=I32), k_pages=PAGES, v_pages=PAGES)
DECODE = dict(q=cpu(2, 4, 64, dtype=BF), k_pages=PAGES, v_pages=PAGES, block_table=cpu(2, 2, dtype=I32),
              seq_lens=cpu(2, dtype=I32), out=cpu(2, 4, 64, dtype=BF),
              workspace=cpu(1 << 20, dtype=torch.uint8))
SCORES = dict(q=cpu(5, 4, 64, dtype=BF), k=cpu(5, 2, 64, dtype=BF), lse=cpu(5, 4), q_offsets=cpu(2, dtype=I32),
              k_offsets=cpu(2, dtype=I32), score_out=cpu(1, 2, 5), max_q_len=5, max_k_len=5)
EVICT = dict(budget=4, recent=1, k_pages=PAGES, v_pages=PAGES, block_table=cpu(2, 2, dtype=I32),
             seq_lens=cpu(2, dtype=I32), score=cpu(2, 2, 30), dst_table=cpu(2, 1, dtype=I32), k_dst=PAGES,
             v_dst=PAGES, kept=cpu(2, 2, 4, dtype=I32), new_lens=cpu(2, dtype=I32),
             workspace=cpu(4096, dtype=torch.uint8))


@pytest.fixture
def on_gpu(monkeypatch):
    """Tensors of the CPU pass for tensors of device 0, and nothing is launched."""
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(q, "_on_device", lambda *a: pytest.fail("the call was made"))


def calls():
    return [(lambda **a: q.paged_kv_append(DESC, **a), APPEND),
            (lambda **a: q.paged_decode_attn(DESC, **a), DECODE),
            (q.attn_scores, SCORES), (lambda **a: q.paged_kv_evict(DESC, **a), EVICT)]


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("bad", [None, 3, [1, 2], "x"])
def test_not_a_tensor(which, bad, on_gpu):
    call, good = calls()[which]
    for name, value in good.items():
        if not isinstance(value, torch.Tensor) or (name == "workspace" and bad is None):
            continue
        with pytest.raises(TypeError, match=f"{name}: expected a tensor"):
            call(**{**good, name: bad})


@pytest.mark.parametrize("which", range(4))
def test_other_dimensions(which, on_gpu):
    call, good = calls()[which]
    for name, value in good.items():
        if isinstance(value, torch.Tensor):
            for shape in ((), (3,), (1, 1, 1, 1, 1)):
                if len(shape) == value.dim():
                    continue
                with pytest.raises(ValueError, match=f"{name}: shape"):
                    call(**{**good, name: cpu(*shape).to(value.dtype)})


def test_optional_tensors(on_gpu):
    for name in ("lse", "score_out"):
        with pytest.raises(TypeError, match=f"{name}: expected a tensor"):
            q.paged_decode_attn(DESC, **DECODE, **{name: 7})
    with pytest.raises(TypeError, match="score_in: expected a tensor"):
        q.paged_decode_attn(DESC, **DECODE, score_out=cpu(2, 2, 30), score_in=7)
    with pytest.raises(TypeError, match="score_in: expected a tensor"):
        q.attn_scores(**SCORES, score_in=[0.0])
    with pytest.raises(TypeError, match="new_offsets: expected a tensor"):
        q.paged_kv_append(DESC, **APPEND, new_offsets=[0, 1, 2])
    with pytest.raises(TypeError, match="score_out: expected a tensor"):
        q.paged_kv_evict(DESC, **EVICT, score_out=1)
    codes = q.make_paged_desc(2, 30, 8, 16, 2, 4, 2, 64, kv_fp8=True)
    with pytest.raises(TypeError, match="k_scale: expected a tensor"):
        q.paged_decode_attn(codes, **DECODE, k_scale=1.0, v_scale=1.0)


@pytest.mark.parametrize("big", [1 << 31, 1 << 32, (1 << 32) + 4, -(1 << 31) - 1])
def test_numbers_past_32_bits(big, on_gpu):
    for name in ("window", "max_q_len", "max_k_len"):
        with pytest.raises(ValueError, match=name):
            q.attn_scores(**{**SCORES, name: big})
    for name in ("budget", "recent"):
        with pytest.raises(ValueError, match=name):
            q.paged_kv_evict(DESC, **{**EVICT, name: big})
    with pytest.raises(ValueError, match="dst_num_pages"):
        q.paged_evict_workspace_size(DESC, big)
    names = ("num_seqs", "max_seq_len", "num_pages", "page_size", "max_pages_per_seq", "num_q_heads",
             "num_kv_heads", "head_dim")
    for i, name in enumerate(names):
        sizes = [2, 30, 8, 16, 2, 4, 2, 64]
        sizes[i] = big
        with pytest.raises(ValueError, match=name):
            q.make_paged_desc(*sizes)


def test_without_private_names():
    """A PyTorch that has no such names: the module loads, and its host-side parts work."""
    code = ("import torch\n"
            "for n in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    hasattr(torch._C, n) and delattr(torch._C, n)\n"
            "class S: cuda_stream = 77\n"
            "torch.cuda.current_stream = lambda i: S if i == 3 else None\n"
            "torch.cuda.current_device = lambda: 3\n"
            "import prefill_only_cascade_gb300 as q\n"
            "assert q.paged_decode_workspace_size(q.make_paged_desc(2, 30, 8, 16, 2, 4, 2, 64)) > 0\n"
            "got = []\n"
            "q._on_device(lambda *a: got.append(a) or 0, 'x', 3, None, 1, 2)\n"
            "assert got == [(1, 2, 77)], got\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=240)
    assert run.returncode == 0, run.stderr
