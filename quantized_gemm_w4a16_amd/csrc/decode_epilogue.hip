// decode_epilogue.hip -- the decode kernels of decode.hip with bias, activation
// (plain or gated pair) and residual in their epilogue (gfx950).
#define SPEAR_EPILOGUE 1
#include "decode.hip"
