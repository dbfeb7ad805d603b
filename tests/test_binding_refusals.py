"""What the Python calls refuse before the library sees it: memory and sizes
that a kernel would misread."""
import pytest
import torch

import block_causal_relu_b200 as lcla

BF = torch.bfloat16


def test_a_workspace_on_the_host_is_refused():
    with pytest.raises(TypeError):
        lcla._workspace(torch.zeros(1 << 16, dtype=torch.uint8), 1 << 10, torch.device("cuda", 0))
    with pytest.raises(TypeError):
        lcla._workspace(1 << 26, 1 << 10, torch.device("cuda", 0))
    assert lcla._workspace(None, 0, torch.device("cuda", 0)) == (None, 0)


@pytest.mark.gpu
def test_workspaces_of_every_call():
    q = torch.randn(1, 2000, 2, 32, device="cuda").to(BF)
    g = torch.zeros(1, 2000, 2, device="cuda")
    c, s = lcla.rotary_tables(2000, 32)
    w = torch.ones(32, device="cuda")
    state = torch.zeros(1, 2, 33, 32, device="cuda")
    blocks = torch.tensor([0, 800, 2000], dtype=torch.int32, device="cuda")
    total, ws = lcla.shard_begin(q, q, c, s, 500)
    calls = [lambda x: lcla.forward(q, q, q, c, s, 500, workspace=x),
             lambda x: lcla.forward_blocks(q, q, q, c, s, blocks, workspace=x),
             lambda x: lcla.step(q, q, q, c, s, state, False, workspace=x),
             lambda x: lcla.shard_begin(q, q, c, s, 500, workspace=x),
             lambda x: lcla.qk_norm_rope_backward(q, q, q, q, c, s, q_weight=w, k_weight=w, workspace=x),
             lambda x: lcla.gated_forward(q, q, q, g, workspace=x),
             lambda x: lcla.gated_step(q, q, q, g, torch.zeros(1, 2, 32, 32, device="cuda"), False, workspace=x),
             lambda x: lcla.gated_backward(q, q, q, q, g, workspace=x)]
    with pytest.raises(TypeError):
        lcla.shard_end(q, q, q, c, s, 500, total[None], 0, ws.cpu())
    for call in calls:
        with pytest.raises(TypeError):
            call(torch.zeros(1 << 24, dtype=torch.uint8))
        with pytest.raises(ValueError):
            call(torch.zeros(1 << 24, 2, dtype=torch.uint8, device="cuda")[:, 0])
        call(torch.empty(1 << 22, dtype=torch.float32, device="cuda"))     # bytes count, not elements


@pytest.mark.parametrize("kw", [dict(n=(1 << 32) + 5), dict(n=1 << 31), dict(dims=[(1 << 32) + 32]), dict(first=1 << 63),
                                dict(first=(1 << 64) + 3), dict(first=-(1 << 64)),
                                dict(dims=[8, 8], extents=[(1 << 32) + 7])])
def test_sizes_that_do_not_fit_the_library_are_refused(kw):
    """ctypes passes them modulo 2^32 (2^64): a table of other positions, or of other sizes."""
    a = dict(n=4, dims=[32])
    a.update(kw)
    with pytest.raises(lcla.LclaError):
        lcla.rotary_tables(a.pop("n"), a.pop("dims"), **a)


@pytest.mark.gpu
def test_tensors_of_more_tokens_than_an_int_holds():
    """2^31 + 5 rows of 8 entries (34 GB), in place: not taken for fewer of them."""
    if torch.cuda.mem_get_info()[0] < 50e9:
        pytest.skip("needs 50 GB")
    q = torch.empty(1, (1 << 31) + 5, 1, 8, device="cuda", dtype=BF)
    c, s = lcla.rotary_tables(64, 8)
    at = torch.zeros(1, 1, dtype=torch.int64, device="cuda").expand(1, (1 << 31) + 5)
    with pytest.raises(lcla.LclaError):
        lcla.qk_norm_rope(q, None, c, s, positions=at, out=(q, None))
    with pytest.raises(lcla.LclaError):
        lcla.qk_norm_rope_backward(q, None, q, None, c, s, positions=at, out=(q, None))


def test_tables_on_the_host_are_refused():
    """Not made on the current CUDA device instead."""
    for kw in (dict(), dict(stream=0)):
        with pytest.raises(ValueError):
            lcla.rotary_tables(4, 32, device="cpu", **kw)
