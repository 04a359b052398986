"""Which tile shape each product of the dense block and of the 8-bit integer products
takes at the sizes that the GPU tests run: all of the shapes, so that none is built that no
test has seen.  The rule itself (csrc/moe_tile.hpp, csrc/moe_dense_grad.hip) is compiled for
the host and asked."""
import os
import subprocess

import pytest

from bit_block_quantized_nvfp4_amd import build as b

PROGRAM = r"""
#include "moe_dense_grad.hip"
#include <cstdio>
int main() {
  using namespace moe;
  char kind;
  int t, n, k;
  printf("%d\n", kTileShapes16);
  while (scanf(" %c %d %d %d", &kind, &t, &n, &k) == 4) {
    if (kind == 'd')  // T, H, I: gate_up, down, dh, the three gradients
      printf("%d %d %d %d\n", tile_shape(t, 2 * k, steps_of(n, 2)), tile_shape(t, n, steps_of(k, 2)),
             tile_shape(t, k, steps_of(n, 2)), grads_shape(grads_of(t, n, k)));
    else  // T, N, K of an integer product
      printf("%d\n", tile_shape(t, n, steps_of(k, 1)));
  }
}
"""
STREAMED = 16  # rows up to which forward products stream their weights


@pytest.fixture(scope="module")
def shapes(tmp_path_factory):
    """(number of shapes, function from [(kind, a, b, c)] to tuples of shapes)"""
    try:
        cc = b.hipcc()
    except RuntimeError:
        pytest.skip("needs hipcc")
    d = tmp_path_factory.mktemp("choice")
    (d / "choice.hip").write_text(PROGRAM)
    # the launches need the rest of the library; the program does not call them
    subprocess.run([cc, f"--offload-arch={b.ARCH}", "--cuda-host-only", "-std=c++17", "-w", "-I", b.CSRC,
                    str(d / "choice.hip"), "-o", str(d / "choice"), "-Wl,--unresolved-symbols=ignore-all"],
                   check=True, capture_output=True)

    def ask(sizes):
        text = "".join("%s %d %d %d\n" % s for s in sizes)
        out = subprocess.run([str(d / "choice")], input=text, capture_output=True, text=True, check=True).stdout
        lines = [tuple(map(int, ln.split())) for ln in out.splitlines()]
        assert len(lines) == len(sizes) + 1
        return lines[0][0], lines[1:]

    return ask


def _parameters(test, names):
    return [v for m in test.pytestmark if m.name == "parametrize" and m.args[0] == names for v in m.args[1]]


@pytest.mark.slow
def test_every_shape_of_the_block_is_run(shapes):
    import test_gpu_dense_shapes as t

    n, got = shapes([("d", *s) for s in t.FORWARD if s[0] > STREAMED])
    assert all({g[i] for g in got} == set(range(n)) for i in (0, 1))
    n, got = shapes([("d", *s) for s in t.GRADIENTS])
    assert all({g[i] for g in got} == set(range(n)) for i in (2, 3))


@pytest.mark.slow
def test_every_shape_of_the_integer_products_is_run(shapes):
    import test_gpu_dense_chain as chain
    import test_gpu_int8 as t

    both = _parameters(chain.test_other_tiles_of_the_products_in_8_bits, "T,N,K")
    for own in (t.LINEAR, _parameters(t.test_gated, "T,N,K")):
        n, got = shapes([("i", *s) for s in own + both if s[0] > STREAMED])
        assert {g[0] for g in got} == set(range(n))


def test_every_stream_of_the_forward_pass_is_run():
    """Up to 16 rows: tiles of 8 weight rows, and of 16 with K on both sides of 4096 (down)."""
    import test_gpu_dense_shapes as t

    few = [s for s in t.FORWARD if s[0] <= STREAMED]
    assert {T <= 8 and I <= 4096 for T, H, I in few} == {False, True}
    assert {0 if T <= 8 and H <= 2048 else 1 if I < 4096 else 2 for T, H, I in few} == {0, 1, 2}
