import gc
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU")


def pytest_collection_finish(session):
    gc.collect()
    gc.freeze()  # what the imports made is not looked through again, so that the collection below is quick


def pytest_runtest_setup(item):
    # A test that catches an error keeps itself, and a graph it captured, in a cycle (the error's traceback holds its frame).
    # Collected while another test captures, that graph's end would be an error inside a destructor: it goes here.
    if item.get_closest_marker("gpu"):
        gc.collect()


def golden_path(name: str) -> str:
    return os.path.join(ROOT, "tests", "golden", name)


def read_golden_examples(name: str):
    """Parse 'key: values' blocks separated by blank lines."""
    blocks, cur = [], {}
    for line in open(golden_path(name)):
        line = line.rstrip("\n")
        if line.startswith("#"):
            continue
        if not line.strip():
            if cur:
                blocks.append(cur)
                cur = {}
            continue
        k, v = line.split(":", 1)
        cur[k.strip()] = v.strip()
    if cur:
        blocks.append(cur)
    return blocks
