"""The generation entry points refuse bad arguments on the host, before touching CUDA."""
import ctypes

import pytest
import torch

INVALID, ALIGN, WS = 1, 2, 4
HUGE = 2 ** 31


@pytest.fixture(scope="module")
def L():
    from lm_head_top_tcgen05_gb300 import build
    from lm_head_top_tcgen05_gb300._lib import lib

    build.build()
    return lib()


def test_quantize_is_checked(L):
    def call(x=16, t=0, rows=4, cols=64, ld=64, q=16, s=16):
        return L.fkl_quantize_int8(x, t, rows, cols, ld, q, s, None)

    assert call(t=3) == INVALID and call(t=-1) == INVALID
    assert call(rows=-1) == INVALID and call(rows=HUGE) == INVALID
    assert call(cols=0) == INVALID and call(ld=63) == INVALID
    assert call(x=None) == INVALID and call(q=None) == INVALID and call(s=None) == INVALID
    assert call(x=18) == ALIGN and call(s=18) == ALIGN
    assert call(x=17, t=1) == ALIGN


def test_workspace_sizes(L):
    for f in (L.fkl_int8_matmul_workspace_size, L.fkl_int8_linear_workspace_size):
        assert f(1, 1, 16) >= 256 and f(0, 5, 64) >= 256
        assert f(4096, 201088, 2880) >= 256
        assert f(4, 10, 40) == 0          # K not a multiple of 16
        assert f(4, 10, 0) == 0 and f(4, 0, 64) == 0 and f(-1, 10, 64) == 0
        assert f(4, 10, 131072) > 0 and f(4, 10, 131088) == 0
        assert f(HUGE, 10, 64) == 0 and f(4, HUGE, 64) == 0


def test_products_are_checked(L):
    def call(M=4, N=10, K=64, x=16, xs=16, w=16, ws=16, t=0, out=16, ldo=10, work=256, n=1 << 30):
        return L.fkl_int8_matmul(x, xs, w, ws, M, N, K, t, out, ldo, work, n, None)

    def linear(M=4, N=10, K=64, x=16, xt=1, ldx=64, w=16, ws=16, t=0, out=16, ldo=10, work=256, n=1 << 30):
        return L.fkl_int8_linear(x, xt, ldx, w, ws, M, N, K, t, out, ldo, work, n, None)

    for f in (call, linear):
        assert f(t=9) == INVALID and f(K=72) == INVALID and f(M=-1) == INVALID and f(N=0) == INVALID
        assert f(ldo=9) == INVALID
        for name in ("x", "w", "ws", "out"):
            assert f(**{name: None}) == INVALID, name
        assert f(w=24) == ALIGN and f(ws=18) == ALIGN and f(out=18) == ALIGN
        assert f(work=None) == WS and f(n=8) == WS and f(work=128) == ALIGN
    assert call(x=24) == ALIGN and call(xs=None) == INVALID
    assert linear(xt=5) == INVALID and linear(ldx=63) == INVALID and linear(x=17) == ALIGN


def test_sample_is_checked(L):
    from lm_head_top_tcgen05_gb300._lib import FklSampleParams

    def call(x=16, t=0, B=4, V=100, ld=100, u=16, p=None, tok=16, lp=16):
        p = FklSampleParams() if p is None else p
        return L.fkl_sample(x, t, B, V, ld, u, ctypes.byref(p), tok, lp, None)

    assert call(t=3) == INVALID and call(B=-1) == INVALID and call(B=HUGE) == INVALID
    assert call(V=0) == INVALID and call(V=2 ** 22 + 1, ld=2 ** 23) == INVALID and call(ld=99) == INVALID
    assert call(x=None) == INVALID and call(u=None) == INVALID and call(tok=None) == INVALID
    assert call(x=18) == ALIGN and call(x=17, t=2) == ALIGN and call(u=18) == ALIGN
    assert call(p=FklSampleParams(top_k_rows=18)) == ALIGN
    assert L.fkl_sample(16, 0, 4, 100, 100, 16, None, 16, 16, None) == INVALID


def test_params_struct_layout_matches_header(tmp_path):
    import subprocess
    from pathlib import Path

    from lm_head_top_tcgen05_gb300._lib import FklSampleParams

    root = Path(__file__).resolve().parent.parent
    fields = [f[0] for f in FklSampleParams._fields_]
    src = tmp_path / "t.c"
    src.write_text('#include <stdio.h>\n#include "fkl_generate.h"\nint main(void) {\n'
                   + "".join(f'printf("%zu\\n", offsetof(fkl_sample_params, {f}));\n' for f in fields)
                   + 'printf("%zu\\n", sizeof(fkl_sample_params)); return 0; }\n')
    subprocess.run(["gcc", "-I", str(root / "include"), str(src), "-o", str(tmp_path / "t")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "t")], capture_output=True, text=True).stdout.split()]
    assert got == [getattr(FklSampleParams, f).offset for f in fields] + [ctypes.sizeof(FklSampleParams)]


def test_binding_needs_cuda_tensors():
    import lm_head_top_tcgen05_gb300 as fkl

    with pytest.raises(ValueError):
        fkl.quantize_int8(torch.zeros(2, 16))
    with pytest.raises(ValueError):
        fkl.int8_linear(torch.zeros(2, 16), torch.zeros(3, 16, dtype=torch.int8), torch.zeros(3))
    with pytest.raises(ValueError):
        fkl.sample(torch.zeros(2, 16), torch.zeros(2))


def _function(source, name):
    """The text of a device function's body."""
    at = source.index("{", source.index(f" {name}("))
    depth, end = 0, at
    while depth > 0 or end == at:
        depth += {"{": 1, "}": -1}.get(source[end], 0)
        end += 1
    return source[at:end]


@pytest.mark.parametrize("role", ["i8_convert", "i8_mma", "i8_epilogue"])
def test_waits_of_whole_warps_have_one_answer(role):
    # Lanes that leave a wait with different answers part for good, and the launch hangs at the next
    # warp barrier; it takes a wait that runs out just as its barrier completes, so it is read here.
    from pathlib import Path

    body = _function((Path(__file__).resolve().parent.parent / "lm_head_top_tcgen05_gb300" / "csrc"
                      / "fkl_int8_gemm.cu").read_text(), role)
    body = body.replace("mbar_wait_drain(", "")  # made by the one lane that issues
    assert "warp_wait(" in body and "mbar_wait" not in body


def test_threads_do_not_share_a_default_workspace(monkeypatch):
    # the two launches of a product hand data over in it, and another thread's may come between
    import threading

    from lm_head_top_tcgen05_gb300 import generate

    cpu, got, both = torch.device("cpu"), {}, threading.Barrier(2)
    monkeypatch.setattr(generate, "_capturing", lambda: False)  # no driver to ask here

    def work(name):
        first = generate._workspace(1000, cpu, 7, None)
        both.wait()
        got[name] = first, generate._workspace(500, cpu, 7, None), generate._workspace(500, cpu, 8, None)
        both.wait()

    threads = [threading.Thread(target=work, args=(n,)) for n in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for first, again, other in got.values():
        assert first.numel() >= 1000 and again.data_ptr() == first.data_ptr() != other.data_ptr()
    assert got[0][0].data_ptr() != got[1][0].data_ptr()


def test_captured_calls_do_not_keep_the_default_workspace(monkeypatch):
    # a graph records its workspace's address, and a later call may drop the thread's buffer for a larger
    from lm_head_top_tcgen05_gb300 import generate

    cpu, capturing = torch.device("cpu"), [False]
    monkeypatch.setattr(generate, "_capturing", lambda: capturing[0], raising=False)
    eager = generate._workspace(1000, cpu, 9, None)
    capturing[0] = True
    captured = generate._workspace(1000, cpu, 9, None)
    other = generate._workspace(1000, cpu, 9, None)
    assert captured.numel() >= 1000 and len({t.data_ptr() for t in (eager, captured, other)}) == 3
    capturing[0] = False
    assert generate._workspace(1000, cpu, 9, None).data_ptr() == eager.data_ptr()


def test_late_tokens_hook_is_checked(L):
    def call(M=5, N=10, K=64, limit=2 * 10 ** 6, late=10 ** 6, ldo=10):
        return L.fkl_test_int8_matmul_late(16, 16, 16, 16, M, N, K, 0, 16, ldo, limit, late, 256, 1 << 30, None)

    assert call(M=4) == INVALID and call(M=0) == INVALID     # no tensor cores
    assert call(limit=10 ** 5) == INVALID and call(limit=2 * 10 ** 9) == INVALID
    assert call(late=0) == INVALID and call(late=2 * 10 ** 9) == INVALID
    assert call(ldo=9) == INVALID and call(K=72) == INVALID


def test_read_status_sees_the_default_workspaces(monkeypatch):
    # of the loss and, after it, of the calling thread's last product on the current stream
    import lm_head_top_tcgen05_gb300 as fkl
    from lm_head_top_tcgen05_gb300 import generate

    class Fake:
        def fkl_read_status(self, ptr, stream):
            word = ctypes.cast(ptr, ctypes.POINTER(ctypes.c_uint32))[0]
            return {0: 0, 1: 6, 4: 8}[word]

    cpu = torch.device("cpu")
    monkeypatch.setattr(fkl, "lib", Fake)
    monkeypatch.setattr(fkl, "_stream", lambda device: None)
    monkeypatch.setattr(fkl, "_default_ws", {})
    monkeypatch.setattr(generate, "_capturing", lambda: False)
    monkeypatch.setattr(generate, "_stream", lambda device: 31)
    with pytest.raises(KeyError):
        fkl.read_status(device=cpu)
    product = generate._workspace(256, cpu, 31, None).zero_()
    assert fkl.read_status(device=cpu) == 0
    product[0] = 4
    assert fkl.read_status(device=cpu) == 8
    loss = fkl._ws_for(None, 256, cpu).zero_()
    assert fkl.read_status(device=cpu) == 8
    loss[0] = 1
    assert fkl.read_status(device=cpu) == 6
    own = fkl.Workspace(cpu)
    own.get(256, cpu).zero_()
    assert fkl.read_status(own) == 0


def test_bins_of_the_second_histogram_have_one_rounding():
    # three loops of the sampler evaluate it and must agree; the compiler may contract a plain product
    # and sum in one of them and not in another
    import re
    from pathlib import Path

    body = _function((Path(__file__).resolve().parent.parent / "lm_head_top_tcgen05_gb300" / "csrc"
                      / "fkl_sample.cu").read_text(), "fine_bin")
    assert "__fmaf_rn(" in body and "__fmul_rn(" in body and not re.search(r" [+*] ", body)


def test_extents_whose_tiles_pass_32_bits_are_refused(L):
    # the kernels' row and channel numbers are ints, a whole tile beyond the last one included
    most = 2 ** 31 - 512
    for f in (L.fkl_int8_matmul_workspace_size, L.fkl_int8_linear_workspace_size):
        assert f(4, most, 16) > 0 and f(most, 1, 16) > 0
        assert f(4, most + 1, 16) == 0 and f(most + 1, 1, 16) == 0 and f(1, 2 ** 31 - 1, 64) == 0
        assert f(most, most, 16) == 0
    assert L.fkl_int8_matmul(16, 16, 16, 16, 4, 2 ** 31 - 1, 64, 0, 16, 2 ** 31, 256, 1 << 40, None) == INVALID


def test_workspace_holds_partial_sums_only_of_cut_tiles(L):
    # otherwise the header (at most 16 KB), the tokens in fp16 and their scales, each rounded up to 256
    for M, N, K in ((4096, 201088, 2880), (64, 151936, 4096), (203, 50261, 1456), (8192, 4096, 4096)):
        assert L.fkl_int8_linear_workspace_size(M, N, K) <= 16384 + 2 * M * K + 4 * M + 512
    for M, N, K in ((9, 4096, 2880), (16, 4096, 8192), (140, 19500, 8000)):
        assert L.fkl_int8_linear_workspace_size(M, N, K) > 16384 + 2 * M * K + 4 * M + 512


def test_product_reads_nothing_as_constant_data():
    # it starts beside the kernel that writes the tokens and their scales: the path for data that is
    # constant during a launch (__ldg) may give what was there before
    from pathlib import Path

    source = (Path(__file__).resolve().parent.parent / "lm_head_top_tcgen05_gb300" / "csrc" / "fkl_int8_gemm.cu").read_text()
    code = "\n".join(line.split("//")[0] for line in source.splitlines())
    assert "__ldg(" not in code and ".nc." not in code and "__restrict__" not in code
