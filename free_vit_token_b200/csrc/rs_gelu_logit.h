// Generated by gen_gelu_logit.py. GELU(z) = z / (1 + 2^(-z Q(z^2))), Q of degree 9. In
// float32 max |error| / |GELU| 2.3e-06 for z >= -4.4, max |error| 1.8e-08 below.
#pragma once
#define RS_GELU_LOGIT_Q0 2.302214580e+00f
#define RS_GELU_LOGIT_Q1 1.048201286e-01f
#define RS_GELU_LOGIT_Q2 -8.254221336e-05f
#define RS_GELU_LOGIT_Q3 -1.627486627e-04f
#define RS_GELU_LOGIT_Q4 1.162639425e-05f
#define RS_GELU_LOGIT_Q5 -3.228179192e-07f
#define RS_GELU_LOGIT_Q6 -6.224912647e-09f
#define RS_GELU_LOGIT_Q7 7.804179854e-10f
#define RS_GELU_LOGIT_Q8 -2.355645458e-11f
#define RS_GELU_LOGIT_Q9 2.574030254e-13f
