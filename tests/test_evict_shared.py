"""Host-side refusals of the eviction that keeps the shared pages up to date.  CPU only."""
import pytest

from deepseek_v4_sparse_indexer_gb300 import _binding as B
from test_more_abi import EVICT, FAKE, call


@pytest.fixture(scope="module")
def lib():
    return B.load()


def _args():
    args = {}
    for k, v in EVICT.items():
        args[k] = v
        if k == "n_shared":
            args[k], args["n_shared_out"] = FAKE, FAKE
    return args


@pytest.mark.parametrize("change", [dict(n_shared=None), dict(n_shared_out=None), dict(n_shared=None, n_shared_out=None),
                                    dict(mass=None), dict(gone=FAKE), dict(limit=99), dict(keep=0), dict(page_size=4)])
def test_evict_shared_rejects(lib, change):
    assert call(lib.ds4a_paged_evict_shared, _args(), **change) == B.DS4A_EINVAL


def test_evict_shared_workspace_and_types(lib):
    assert call(lib.ds4a_paged_evict_shared, _args(), ws=None) == B.DS4A_EWORKSPACE
    assert call(lib.ds4a_paged_evict_shared, _args(), rows_type=B.DS4A_F16) == B.DS4A_EUNSUPPORTED


def test_injected_error(lib):
    lib.ds4a_debug_inject_error(B.DS4A_ECUDA)
    assert call(lib.ds4a_paged_evict_shared, _args()) == B.DS4A_ECUDA
