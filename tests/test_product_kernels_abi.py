"""The hook that forces a kernel of the experts' products, without a GPU."""
from lsd_radix_sort_pass_amd import _lib


def test_product_kernel_hook():
    lib = _lib.load()
    prev = lib.rs_prof_product_kernel(_lib.RS_PRODUCT_WIDE)
    try:
        assert lib.rs_prof_product_kernel(5) == _lib.RS_PRODUCT_WIDE
        assert lib.rs_prof_product_kernel(-1) == 0 and lib.rs_prof_product_kernel(0) == 0
    finally:
        lib.rs_prof_product_kernel(prev)
