"""dsa_mla_prefill and the page operators allocate no device memory, whatever their sizes (first calls in a
process aside, which load kernels): the device's free memory is what it was."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mla_paged_gb300 import build
    build.build()
    import sparse_mla_paged_gb300.api as api
    api.step_device_status()
    return api


def test_nothing_is_allocated(api):
    def ints(*v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def make(n, rows, heads, blocks):
        pages = 2 * n * blocks + 9
        z = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
        tables = torch.arange(2 * n * blocks, dtype=torch.int32, device="cuda").view(2 * n, blocks)
        q, cache = z(rows, heads, 512, dtype=torch.bfloat16), z(pages, 64 * 512, dtype=torch.uint8)
        shares, free, info = z(pages), torch.arange(pages, dtype=torch.int32, device="cuda"), z(4)
        return dict(q=q, cache=cache, tables=tables, blocks=blocks, base=ints(*[64 * blocks - 8] * n), new=ints(*[rows // n] * n), heads=heads,
                    out=torch.empty_like(q), ws=api.alloc_prefill_workspace(n, rows, heads), pws=api.alloc_pages_workspace(pages),
                    shares=shares, free=free, count=ints(9), info=info, lens=ints(*[64 * blocks - 8] * (2 * n)), keeps=ints(*[40] * (2 * n)),
                    parents=ints(*range(n)), children=ints(*range(n, 2 * n)))

    def calls(s):
        api.prefill(s["q"], s["cache"], s["cache"], s["tables"][:len(s["base"])], s["blocks"], s["base"], s["new"], s["heads"], 64, 64 * 512, 1.0, 1.0,
                    0.1, out=s["out"], workspace=s["ws"])
        api.copy_pages([s["cache"]], s["parents"], s["children"])
        api.fork_pages([s["cache"]], s["parents"], s["children"], s["lens"], 64, s["tables"], s["free"], s["shares"], info=s["info"],
                       workspace=s["pws"])
        api.release_pages(s["tables"], s["lens"], s["keeps"], 64, s["shares"], s["free"], s["count"], info=s["info"], workspace=s["pws"])
        api.compact_pages([s["cache"]], s["tables"], s["keeps"], 64, s["shares"], s["free"], s["count"], info=s["info"], workspace=s["pws"])

    small, large = make(2, 6, 16, 3), make(40, 320, 64, 50)
    calls(small)
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0], torch.cuda.memory_reserved()
    for s in (large, small, large):
        calls(s)
    torch.cuda.synchronize()
    assert (torch.cuda.mem_get_info()[0], torch.cuda.memory_reserved()) == before
