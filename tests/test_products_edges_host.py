"""Products on decoded weights, what can be shown without a GPU: how their
sources load, what the binding does at its edges."""
import ctypes
import glob
import os
import re

import pytest
import torch
from torch.autograd import forward_ad

import trellis_coded_weight_bitshift_b200 as tcq
from trellis_coded_weight_bitshift_b200 import _abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "trellis_coded_weight_bitshift_b200", "csrc")


def _code(path):
    """A source without its comments."""
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)


def test_kernels_that_start_early_use_no_read_only_loads():
    # a kernel launched by tcq_launch.cuh runs while its predecessor still writes: no load of its may be one that
    # the compiler takes for constant (and moves above the wait), in its source or in a header that it includes
    early = [p for p in glob.glob(os.path.join(CSRC, "*.cu")) if '"tcq_launch.cuh"' in open(p).read()]
    assert len(early) >= 2
    headers = [os.path.join(CSRC, h) for h in ("tcq_launch.cuh", "tcq_tensor.cuh", "tcq_activation.cuh")]
    for path in early + headers:
        code = _code(path)
        found = re.findall(r"__ldg\b|ld\.global\.nc|const\s+\w+\s*\*\s*(?:const\s+)?__restrict__\s*\w+", code)
        assert not found, (path, found)


def test_every_kernel_waits_before_it_lets_the_next_start():
    # the next kernel may start once all blocks have called let_next_start: after their own wait, not before
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        if '"tcq_launch.cuh"' not in open(path).read():
            continue
        for body in re.split(r"\n__global__", _code(path))[1:]:
            body = body.split("\n}\n")[0]
            assert 0 <= body.find("after_previous()") < body.find("let_next_start()"), (path, body[:120])


def test_time_in_which_a_kernel_did_not_run_is_not_waited(tmp_path):
    # a wait's clock goes on while another process has the GPU: two looks seconds apart are no wait of seconds
    from native import compiled
    lib = compiled("waits", tmp_path)

    def over(at, limit):
        got = (ctypes.c_int * len(at))()
        lib.waited((ctypes.c_ulonglong * len(at))(*at), len(at), ctypes.c_ulonglong(limit), got)
        return list(got)[1:]
    ms, s = 10 ** 6, 10 ** 9
    looks = [i * 32 * ms for i in range(80)]                       # a look every 32 ms
    assert over(looks, 2 * s) == [i * 32 * ms > 2 * s for i in range(1, 80)]
    held = [0, 32 * ms, 10 * s, 10 * s + 32 * ms, 10 * s + 64 * ms]
    assert not any(over(held, 2 * s))
    assert over([i * 60 * s for i in range(43)], 2 * s) == [False] * 40 + [True, True]      # and it does end


def test_aborted_products_wait_for_what_is_in_flight():
    # where a wait gives up, the thread that loads drains its loads and the thread that multiplies its products
    code = _code(os.path.join(CSRC, "tcq_product.cu"))
    for name, drains in (("pair_kernel(", ("full + 8 * s", "acc_full + 8 *")), ("rows_kernel(", ("full + 8 * s", "acc_full, 0"))):
        body = code[code.index("    " + name):].split("\n}\n")[0]
        for what in drains:
            assert f"mbar_drain({what}" in body, (name, what)
        # no wait of a thread that issues work is left without a way there
        assert not re.search(r"mbar_wait\((?:full|empty|acc_empty)[^;{]*\)\) break;", body)


def test_every_product_asks_whether_an_earlier_one_gave_up():
    code = _code(os.path.join(CSRC, "tcq_product.cu"))
    for head in ("static tcq_status_t product(", 'extern "C" tcq_status_t tcq_gated_ffn_backward('):
        body = code[code.index(head):].split("\n}\n")[0]
        asks = body.index("if (take_note(note)) return TCQ_ERR_TIMEOUT;")
        assert asks < body.index("make_copies(") and ".note = note;" in body
    assert code.count("if (threadIdx.x == 0 && stop) say_gave_up(p.note);") == 2          # both kernels' last words
    assert "gave up" in _abi.status_string(_abi.TCQ_ERR_TIMEOUT)


# ------------------------------------------------------------------ binding

@pytest.fixture
def on_host(monkeypatch):
    """The binding with host tensors for device ones and torch for the launches."""
    monkeypatch.setattr(tcq, "_require_cuda", lambda *t: None)
    monkeypatch.setattr(tcq, "_empty", lambda shape, dtype: torch.zeros(shape, dtype=dtype))
    monkeypatch.setattr(tcq, "_launch_ffn", lambda x, g, u, act, sizes, out, gate, up, ws: out.copy_((x @ g.t()) * (x @ u.t())))
    monkeypatch.setattr(tcq, "_launch_ffn_backward", lambda x, g, u, gate, up, h, act, sizes, need, ws: tuple(
        torch.ones_like(t) if n else None for t, n in zip((x, g, u), need)))


def _operands():
    g = torch.Generator().manual_seed(0)
    return [torch.randn(s, 6, generator=g).half() for s in (3, 5, 5)]


@pytest.mark.parametrize("grad_mode", [True, False])
@pytest.mark.parametrize("which", [0, 1, 2])
def test_tangents_are_refused_not_lost(on_host, grad_mode, which):
    # the block has no forward-mode rule: a dual operand raises, under no_grad() as well, which leaves forward mode on
    ops = _operands()
    with forward_ad.dual_level(), torch.set_grad_enabled(grad_mode):
        ops[which] = forward_ad.make_dual(ops[which], torch.ones_like(ops[which]))
        with pytest.raises(RuntimeError, match="jvp"):
            tcq.GatedFfn.apply(*ops, tcq.ACT_RELU)


def test_the_block_saves_only_what_a_backward_pass_needs(on_host):
    x, g, u = _operands()
    g.requires_grad_()
    h = tcq.GatedFfn.apply(x, g, u)
    assert h.requires_grad and torch.autograd.grad(h.sum(), g)[0].shape == g.shape
    with torch.no_grad():
        assert not tcq.GatedFfn.apply(x, g, u).requires_grad
    assert not tcq.GatedFfn.apply(x, g.detach(), u).requires_grad
    saved = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: saved.append(t) or t, lambda t: t), torch.no_grad():
        tcq.GatedFfn.apply(x, g, u)
    assert not saved


@pytest.mark.parametrize("which,change", [(0, lambda t: t[:2]), (1, lambda t: t[:, :5].contiguous()), (2, lambda t: t.float()),
                                          (3, lambda t: t.half()), (3, lambda t: t[:8].clone())])
def test_the_backward_pass_checks_what_it_is_given_back(on_host, which, change):
    # the kernels take addresses: a saved tensor that comes back smaller, or of another type, must not reach them
    count = iter(range(4))
    leaves = [t.requires_grad_() for t in _operands()]
    with torch.autograd.graph.saved_tensors_hooks(lambda t: (next(count), t), lambda p: change(p[1]) if p[0] == which else p[1]):
        h = tcq.GatedFfn.apply(*leaves)
    with pytest.raises(ValueError):
        h.sum().backward()


def test_pair_instructions_run_only_while_both_blocks_are_there():
    # tensor memory of a pair of blocks is allocated and freed by both: each between two cluster barriers, so that
    # the other block has started and not left
    code = _code(os.path.join(CSRC, "tcq_product.cu"))
    body = code[code.index("    pair_kernel("):].split("\n}\n")[0]
    marks = [m.group(1) for m in re.finditer(r"\b(cluster_sync|tmem_alloc_pair|tmem_dealloc_pair|mma<I8, true>|mma_commit_pair|"
                                             r"tma_load_pair|mbar_arrive_at)\(", body)]
    assert marks[:3] == ["cluster_sync", "tmem_alloc_pair", "cluster_sync"]
    assert marks[-3:] == ["cluster_sync", "tmem_dealloc_pair", "cluster_sync"] and marks.count("cluster_sync") == 4
    rows = code[code.index("    rows_kernel("):].split("\n}\n")[0]
    assert not re.search(r"_pair\(|mma<I8, true>", rows)


def test_rht_keeps_converted_signs_until_the_call(monkeypatch):
    # signs of another type are converted for the call; both copies have to live until it has been made
    seen = {}

    class Lib:
        @staticmethod
        def tcq_rht(W, R, C, rows, cols, out, stream):
            for name, at, n in (("rows", rows, R), ("cols", cols, C)):
                seen[name] = list((ctypes.c_float * n).from_address(at))
            return 0
    monkeypatch.setattr(tcq, "lib", lambda: Lib)
    monkeypatch.setattr(tcq, "_require_cuda", lambda *t: None)
    monkeypatch.setattr(tcq, "_stream", lambda: 0)
    for n in (32, 64, 4096):
        rows, cols = torch.ones(n, dtype=torch.int8), -torch.ones(n, dtype=torch.float64)
        tcq.rht(torch.zeros(n, n), rows, cols)
        assert seen["rows"] == [1.0] * n and seen["cols"] == [-1.0] * n


def test_loads_behind_an_early_start_are_fenced():
    # tensor-map loads read what earlier kernels stored: behind the wait, and behind a fence between the two paths
    code = _code(os.path.join(CSRC, "tcq_product.cu"))
    for name, first in (("    pair_kernel(", "tma_load_pair("), ("    rows_kernel(", "load(kb0 + i, i)")):
        body = code[code.index(name):].split("\n}\n")[0]
        assert body.index("after_previous()") < body.index("fence_before_loads()") < body.index(first)
