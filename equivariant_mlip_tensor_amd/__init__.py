"""MI355X-native Clebsch-Gordan tensor-product convolution.

The library is ``libtpconv.so`` (C ABI in ``include/tpconv.h``); ``tpconv``
is its ctypes binding, ``node`` that of the node operators
(``include/tpconv_node.h``).  Build with ``python -m equivariant_mlip_tensor_amd.build``.
"""

__all__ = ["tpconv", "node"]
