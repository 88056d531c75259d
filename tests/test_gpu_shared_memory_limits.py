"""Kernels whose shared memory grows with the call: every size up to the most there
may be works in a process that has made no larger call, and host threads with
calls of different sizes do not disturb one another."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import attention_forward_13_gb300 as A
from tests._parity import no_device_error

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def reserve(B):
    """B sequences of one token each, one page a sequence, all growing by one token."""
    pools = [torch.zeros(B, 16, 1, 8, dtype=torch.float16, device="cuda") for _ in range(2)]
    table, one = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1), i32([1] * B)
    t, l, r, f = A.attn_cache_reserve(*pools, table, one, one, one)
    assert torch.equal(t, table) and l.eq(2).all() and r.eq(1).all() and f.item() == 0


def reorder(B):
    table, one = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1), i32([1] * B)
    t, l, r = A.attn_cache_reorder(table, one, one, torch.arange(B, dtype=torch.int32, device="cuda").flip(0), 16)
    assert torch.equal(t, table.flip(0)) and l.eq(1).all() and r.eq(1).all()


def accept(B):
    pools = [torch.zeros(B, 16, 1, 8, dtype=torch.float16, device="cuda") for _ in range(2)]
    table, one = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1), i32([1] * B)
    l, r = A.attn_cache_accept(*pools, table, one, one, torch.zeros_like(table), one, one)
    assert l.eq(1).all() and r.eq(1).all()


def tree_mask(T):
    parents = torch.arange(-1, T - 1, dtype=torch.int32, device="cuda").view(1, T)
    _, depth = A.attn_tree_mask(parents)
    assert torch.equal(depth[0], torch.arange(T, dtype=torch.int32, device="cuda"))


CALLS = {"reserve": reserve, "reorder": reorder, "accept": accept, "tree_mask": tree_mask}

# Around the 48 KB that a block may have without asking: reserve holds 20 bytes a
# sequence (and a few hundred of its own), re-order and accept 32 KB and 4 a
# sequence, the mask T words a node.
SIZES = [("reserve", n) for n in (2438, 2439, 2448, 2457, 2458, 8192)] + \
        [("reorder", n) for n in (4094, 4095, 4096, 4097, 8192)] + \
        [("accept", n) for n in (4094, 4095, 4096, 4097, 8192)] + \
        [("tree_mask", n) for n in (606, 607, 608, 609, 640, 1024)]


@pytest.mark.parametrize("name,size", SIZES, ids=["%s-%d" % s for s in SIZES])
def test_first_call_of_a_process(name, size):
    code = "import tests.test_gpu_shared_memory_limits as t\nt.CALLS[%r](%d)\nt.no_device_error()" % (name, size)
    run = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]


def test_threads_with_calls_of_different_sizes():
    """Host threads on streams of their own, small and large calls in turn."""
    plan = [("reserve", 8192), ("reserve", 2500), ("reorder", 8192), ("reorder", 4200), ("accept", 8192),
            ("accept", 4200), ("tree_mask", 1024), ("tree_mask", 700)]
    errors, go = [], threading.Barrier(len(plan))

    def run(name, size):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                go.wait()
                for _ in range(60):
                    CALLS[name](size)
        except Exception as e:  # (an assert in a thread would be lost)
            errors.append((name, size, repr(e)))

    threads = [threading.Thread(target=run, args=x) for x in plan]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    no_device_error()
