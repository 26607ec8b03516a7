import pytest


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU and the built CUDA library")


def pytest_collection_modifyitems(config, items):
    """GPU tests are skipped, with a reason, on a machine without a CUDA
    device; on a GPU machine they build and load the CUDA library and fail
    loudly if it is missing."""
    try:
        import torch
        has_gpu = torch.cuda.is_available()
    except ImportError:
        has_gpu = False
    if has_gpu:
        return
    skip = pytest.mark.skip(reason="no CUDA device on this machine")
    for item in items:
        if "gpu" in item.keywords:
            item.add_marker(skip)


@pytest.fixture(scope="session")
def cuda_lib():
    from fully_sharded_state_gb300 import build, capi
    build.build()
    return capi.load()


# modules whose GPU tests run the operators' kernels
_OPERATORS = ("test_layer_norm", "test_linear_cross_entropy", "test_muon", "test_ops_path")


@pytest.fixture(autouse=True)
def no_wait_given_up(request):
    """After every GPU test of the operators: no block gave up a wait."""
    yield
    if "gpu" in request.keywords and request.module.__name__.startswith(_OPERATORS) and "cuda_lib" in request.fixturenames:
        from fully_sharded_state_gb300 import ops_wait_timeouts
        assert ops_wait_timeouts() == 0
