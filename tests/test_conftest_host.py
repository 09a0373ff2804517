"""The suite's own hook: what a GPU test leaves in a cycle is gone before the next one, whatever that is called."""
import gc
import weakref

import pytest

import conftest


class Item:
    def __init__(self, gpu, name):
        self.gpu, self.name = gpu, name

    def get_closest_marker(self, name):
        return self.gpu if name == "gpu" else None


@pytest.mark.parametrize("name", ["test_a_step_in_a_graph", "test_capturing", "test_masks", "test_one_launch"])
def test_cycles_go_before_a_gpu_test(name):
    class Held:
        pass
    gc.disable()
    try:
        held = Held()
        held.self, ref = held, weakref.ref(held)
        del held
        conftest.pytest_runtest_setup(Item(None, name))
        assert ref() is not None
        conftest.pytest_runtest_setup(Item(True, name))
        assert ref() is None
    finally:
        gc.enable()
