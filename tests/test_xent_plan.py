"""How the linear cross entropy is cut (host code, no GPU): every variant is reached by the sizes that the GPU tests run."""
import os
import subprocess

import pytest

from xent_sizes import SIZES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LM = os.path.join(ROOT, "fft_long_convolution_flashconv_amd", "csrc", "lm")

PROGRAM = r"""
#include "xent_plan.h"
#include <stdio.h>
#include <stdlib.h>
using namespace h3c::xent;
int main(int n, char **a) {
    const bool wide = atoi(a[1]);
    for (int i = 2; i + 2 < n; i += 3) {
        const int64_t T = atoll(a[i]), D = atoll(a[i + 1]), V = atoll(a[i + 2]);
        const XentPlan p = plan(T, D, V, wide, true, nullptr);
        const int64_t last = V - (p.pieces - 1) * p.piece, first = p.pieces > 1 ? p.piece : V;
        const auto side = [&](int64_t m) { return wide ? side32(T, m) : side16(T, m); };
        const int64_t kv = wide ? last : ceil_to(last, kSlab16);
        const int64_t f[] = {side(V), side(first), side(last), p.side, p.pieces, p.piece, last, p.ranges,
                             (kv + p.range - 1) / p.range, p.wranges, (int64_t)p.bytes,
                             (int64_t)plan(T, D, V, wide, false, nullptr).bytes};
        for (int64_t v : f) printf("%lld ", (long long)v);
        printf("\n");
    }
}
"""
NAMES = ("forward", "grad", "grad_last", "products", "pieces", "piece", "last", "ranges", "last_ranges", "wranges", "bytes",
         "forward_bytes")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, exe = d / "plan.cpp", d / "plan"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", LM, str(src), "-o", str(exe)], check=True)

    def get(io, sizes):
        args = [str(v) for s in sizes for v in s]
        out = subprocess.run([str(exe), "1" if io == "f32" else "0", *args], check=True, capture_output=True, text=True)
        return [dict(zip(NAMES, map(int, line.split()))) for line in out.stdout.splitlines()]

    return get


@pytest.mark.parametrize("io", list(SIZES))
def test_plans_of_the_tested_sizes(plans, io):
    for (size, want), got in zip(SIZES[io], plans(io, [s for s, _ in SIZES[io]])):
        assert {k: got[k] for k in want} == want, size
        if got["pieces"] > 1:
            assert got["last"] < got["piece"], size


def test_every_variant_is_among_them():
    for io, sides in (("16", {64, 128, 256}), ("f32", {32, 64})):
        for what in ("forward", "grad", "products"):
            assert {p[what] for _, p in SIZES[io]} == sides, (io, what)
        p = [p for _, p in SIZES[io]]
        assert any(q["pieces"] > 1 for q in p) and any(q["pieces"] > 1 and q["ranges"] > 1 for q in p)
        assert any(q["pieces"] > 1 and q["last_ranges"] < q["ranges"] for q in p)
    assert any(q["wranges"] > 1 and q["pieces"] > 1 for _, q in SIZES["16"])


@pytest.mark.parametrize("io", list(SIZES))
def test_workspace_sizes(plans, io):
    """What the entry point asks for is the plan's."""
    import fft_long_convolution_flashconv_amd as pkg

    for size, got in zip([s for s, _ in SIZES[io]], plans(io, [s for s, _ in SIZES[io]])):
        code = pkg.F32 if io == "f32" else pkg.BF16
        assert pkg._size("h3conv_linear_xent_workspace_size", *size, code, 1) == got["bytes"]
        assert pkg._size("h3conv_linear_xent_workspace_size", *size, code, 0) == got["forward_bytes"]
