"""Which stream the binding's calls go to."""
import importlib.util
import sys
import types

import pytest
import torch

import trainable_block_sparse_pool_b200 as T


def _copy(monkeypatch, name):
    spec = importlib.util.spec_from_file_location(name, T.__file__, submodule_search_locations=T.__path__)
    module = importlib.util.module_from_spec(spec)
    monkeypatch.setitem(sys.modules, name, module)
    spec.loader.exec_module(module)
    return module


def test_current_stream_without_the_unwrapped_query(monkeypatch):
    # a torch that lacks the unwrapped query of the current stream: the public one is asked
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=1000 + device))
    assert _copy(monkeypatch, "binding_copy")._raw_stream(3) == 1003


@pytest.mark.gpu
def test_calls_on_a_side_stream_follow_its_work():
    # every tensor is made on the stream that the calls go to, by its current-stream default and by name
    page, h_q, h_kv, d, lens = 16, 4, 2, 64, [100, 30]
    K = torch.randn(sum(lens), h_kv, d, device="cuda").bfloat16()
    q = torch.randn(2, h_q, d, device="cuda").bfloat16()
    outs = []
    torch.cuda.synchronize()
    for named in (False, True):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            pages = torch.zeros(9, h_kv, page, d, device="cuda", dtype=torch.bfloat16)
            table = torch.arange(14, device="cuda", dtype=torch.int32).remainder_(9).view(2, 7).contiguous()
            table[1] = torch.tensor([7, 8, 0, 0, 0, 0, 0], dtype=torch.int32).cuda()
            cache = T.make_paged_cache(pages, torch.zeros_like(pages), table)
            cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
            n, start = cu.diff().contiguous(), torch.zeros(2, dtype=torch.int32, device="cuda")
            ws = torch.empty(T.infllm2_paged_workspace_bytes(cache, h_q), dtype=torch.uint8, device="cuda")
            out, back = torch.empty(2, h_q, d, device="cuda"), [torch.empty_like(K) for _ in range(2)]
            kw = {"stream": side} if named else {}
            T.infllm2_paged_write(cache, K, K, start, cu, **kw)
            T.infllm2_paged_read(cache, *back, cu, **kw)
            T.infllm2_paged_decode_attn(cache, q, n, out, ws, **kw)
        side.synchronize()
        assert torch.equal(back[0], K) and torch.equal(back[1], K)
        outs.append(out)
    assert torch.equal(*outs) and T.infllm2_get_device_status() == 0
