"""The cache operators on pools past 4 GB: pages at the end of a large pool give the
bits that the same rows give in a small one."""
import numpy as np
import pytest
import torch

from cache_ops import layer
from int8_quantized_paged_gb300 import kvq
from int8_quantized_paged_gb300.cache import LayerCache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    torch.cuda.init()


def _run(n_pages: int, table: np.ndarray, w: dict, lens):
    """Every operator once on two sequences whose pages the table names."""
    cfg = kvq.config(**w)
    c = LayerCache(cfg, 2, table.shape[1], n_pages, 600, sinks=4)
    c.set_table(table)
    g = torch.Generator().manual_seed(7)

    def rows(n, heads):
        return torch.randn(n, heads, w["head_dim"], generator=g).half().cuda()

    for b, L in enumerate(lens):
        c.append(rows(L, w["n_kv_heads"]), rows(L, w["n_kv_heads"]), torch.arange(L, dtype=torch.int32, device="cuda"),
                 torch.full((L,), b, dtype=torch.int32, device="cuda"))
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    k, v = c.read(torch.arange(300, dtype=torch.int32, device="cuda"), torch.ones(300, dtype=torch.int32, device="cuda"))
    q = rows(2, w["n_heads"])
    dec = torch.empty_like(q)
    c.append_sink_decode(q, rows(2, w["n_kv_heads"]), rows(2, w["n_kv_heads"]), lt - 1, lt, dec,
                         c.sink_workspace(2, 100), 100)
    qs = rows(150, w["n_heads"])
    outs = []
    for window in (0, 100):
        out = torch.empty_like(qs)
        c.prefill(qs, torch.tensor([0, 50, 150], dtype=torch.int32, device="cuda"), lt, out,
                  c.prefill_workspace(2, 150, window), window)
        outs.append(out)
    torch.cuda.synchronize()
    assert c.status_bits() == 0
    c.close()
    return [k, v, dec] + outs


@pytest.mark.parametrize("key", ["llama8b", "llama8b_f16"])
def test_pages_behind_the_first_four_gigabytes(key):
    w = layer(key, n_heads=32, n_kv_heads=8, act="f16")
    lens = [450, 333]
    pages = np.arange(60, dtype=np.int32).reshape(2, 30)
    far = -(-(5 << 30) // kvq.page_bytes(kvq.config(**w), 0))     # five gigabytes each for K and V
    small = _run(60, pages, w, lens)
    large = _run(far, far - 1 - pages, w, lens)
    for a, b in zip(small, large):
        assert torch.equal(a, b)
